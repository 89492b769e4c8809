// shared.cu -- decode attention for a batch whose requests share prefixes.
//
// What is computed: attn_decode's softmax over the visible keys of each row, where key t of
// request b lies in its own slots for t >= prefix_lens[b] and in those of row
// prefix_rows[b] before.  A softmax over the union of two sets of keys is joined from their
// states: with O, l the weighted sum and the sum of weights 2^(x - M) of a set,
//     out = sum_s 2^(M_s) O_s / sum_s 2^(M_s) l_s.
// The keys in front are common to all rows of a group (neighbouring requests with the same
// row and length), so they are one dense contraction, N R G query rows of a KV head against
// every key, and go to tcgen05 here; the keys behind are each request's own and go to
// attend.cu; shared_merge_kernel joins the parts of both.
//
// GB300 mapping of the shared part.  A group's rows (N requests x R rows x G heads of a KV
// head) are packed into the M dimension of 128-row tiles, 128 / G positions a tile: q viewed
// as {D, heads, positions} gives a tile by one TMA box a 64 dims.  A CTA takes a pair of
// such tiles of one KV head and a range of key tiles (128 keys); the ranges of all (group,
// KV head, pair) fill the SMs once.  Where a group has one tile only, the CTA's two softmax
// warpgroups take every other key tile of it each (with a state each): a lone tile's chain
// product - softmax - product would else leave the tensor cores and the softmax waiting for
// one another (four groups of 30 requests over E4M3 61.3 us, with lone tiles 70; 32 x 4 rows over
// INT8 32.8 and 38.2; where few key tiles are left for an SM it costs a part more, two requests over
// 512 keys 15.6 and 14.8).
//   warps 0, 2   load K and V: TMA boxes of whole runs of keys (a page, or 128 of a linear cache),
//                one a lane; where pages are no multiple of 8 keys, 16-byte cp.async by row
//   warp 1       one thread issues tcgen05.mma: S = Q K^T, O += P V (f16, P from TMEM)
//   warps 4..    bring what is loaded into the form that is multiplied: V of a bf16 cache to
//                f16 times a power of two in place (warps 4..7), 8-bit codes to f16 (exact) from
//                a ring of their own (K warps 4..7, V warps 8..11); values outside the group's range
//                become zeros
//   the last 8   softmax, a thread a row of a tile; weights rounded once to f16 and written
//                over S in TMEM
// The plan is made on the device from lengths, rows and positions, by every CTA for itself
// (a captured graph follows them); CTAs are persistent for batches of more pairs than SMs.
//
// What bounds it.  A pair of tiles (head_dim 128, bf16) takes 1.75 us a key tile, of which its products
// are 1.0: the softmax (S read from TMEM twice, a chain of ~2,100 cycles a tile), V's conversion and the
// loads' issue run beside them, at 48% of the issue slots; 256 requests over 32,768 shared keys, 32/8
// heads: 159 to 164 us, 840 to 870 TFLOP/s, of which ~31 are no key tiles (plan, first and last tiles,
// own keys, merge).  A lone tile takes 1.3 us (its K and V are 7.6 TB/s over all SMs), over codes 1.7 to
// 2.0: four warps widen K and four V, 170 to 300 cycles for each 16 codes of a thread, beside the
// softmax warps.  A step over few keys is a chain: the plan 3 us, the first tiles, the merge 3 us (two
// requests over 512 keys 16.8 us).
//
// Scales of 8-bit caches leave the products as in attend.cu: K's multiplies the scores, V's
// enters the weights' exponent, l sums w / vs.  Weights are held times 2^7 (those down to
// 2^-21 of the largest keep f16's 11 bits).  Values of a bf16 cache have such a scale too, or f16
// would lose them from 2^-14 on: those of a tile are multiplied with a power of two (exactly) and the
// weights of its keys divided by it.  The power of the tile before is tried (of a quarter of the first
// tile at first); where the tile's largest value, which the conversion finds by the way, leaves 2^-4 ..
// 2^15 by it, the tile is read and converted again with its own (256 requests over 32,768 keys 160 us;
// with a first round over every tile 166, without powers of two 152).  A CTA leaves O normalised by the plain sum of its
// weights and held times a power of two of its row, in f16 (2^-11, a quarter of the output's bf16
// half step), and the logarithms of both sums.
#include <cuda.h>
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
namespace shr {

constexpr int kBM = 128;       // rows of a tile (two of them a CTA)
constexpr int kBN = 128;       // keys of a tile
constexpr int kTmemCols = 512;
constexpr float kRescaleLog2 = 8.0f;    // the reference maximum moves past this only
constexpr float kWeightLog2 = 7.0f;     // weights are held times 2^7: at most 2^15
constexpr float kScoreTop = 0x1p24f;    // larger scores are reported (as in attend.cu)
constexpr float kFactorTop = 0x1p90f;
// A tile's values are held times 2^80 at most: 128 weights of 2^15, times that, over 2^24 tiles are
// a finite sum; keys whose weights vanish beside another tile's have less than 2^-53 of its own.
constexpr int kShiftTop = 80;
constexpr float kScaleFloor = 0x1p-64f; // the smallest scale
constexpr float kPartWeight = 0x1p-12f;
constexpr float kSmallest = 0x1p-149f;
constexpr int kMaxBatch = 4096;         // requests: the plan's tables lie in the K and V rings
constexpr int kGroupSteps = 13;         // powers of two of groups, 1 .. kMaxBatch

enum Fmt { kBF16 = 0, kE4M3 = 1, kINT8 = 2 };

// Shared memory: Q tile 0, K, V, codes, in stages of 128 keys.  A load is under way for about
// 2 us, longer than a tile's products, and a stage is taken from its request until its last
// product, so depth is what counts: of five bf16 tiles of 128 dims V, which also waits for its
// conversion and for the weights, has three.  Where there is no Q tile 1 its place is one more K
// stage, or two of codes (as a second tile of converted K it was no faster).
template <int FMT, int HD>
struct Cfg {
    static constexpr bool kCodes = FMT != kBF16;
    static constexpr int kHalves = HD / 64;
    // threads that convert a tensor's tiles: K's and V's codes have warps of their own
    static constexpr int kConv = 128;
    static constexpr int kThreads = 128 + (kCodes ? 2 : 1) * kConv + 256;
    // bf16: the rings that TMA fills; 8-bit: f16 tiles converted from a ring of codes
    static constexpr int kKStages = kCodes ? (HD == 128 ? 1 : 2) : HD == 128 ? 2 : 4;
    static constexpr int kVStages = kCodes ? 2 : HD == 128 ? 3 : 5;
    static constexpr int kRawStages = kCodes ? (HD == 128 ? 4 : 8) : 0;
    static constexpr int kQBytes = kBM * HD * 2;
    static constexpr int kTileBytes = kBN * HD * 2;        // of K or V, 16 bits an element
    static constexpr int kRawBytes = kCodes ? kBN * HD : 0;
    static constexpr int kOffK = kQBytes;
    static constexpr int kOffQ1 = kOffK + kKStages * kTileBytes;
    static constexpr int kOffRaw = kOffQ1 + kQBytes;       // (grows back over Q tile 1)
    static constexpr int kOffV = kOffRaw + kRawStages * kRawBytes;
    static constexpr int kOffBar = kOffV + kVStages * kTileBytes;
    // K is passed on and taken back in parts: whole bf16 tiles, 64 dims of converted codes
    static constexpr int kKSplit = kCodes ? kHalves : 1;
    static constexpr int kKPart = kTileBytes / kKSplit;
    static constexpr int kMaxK = kKStages * kKSplit + (kCodes ? 0 : 1);  // with Q tile 1's place
    static constexpr int kMaxRaw = kCodes ? kRawStages + 2 : 0;
    static constexpr int kNumBars = 3 * kMaxK + 3 * kVStages + 2 * kMaxRaw + 10;
    static constexpr size_t kSmem = 1024 + kOffBar + kNumBars * 8 + 16;
    static_assert(kSmem + 256 <= 227 * 1024, "shared memory");
    // the plan: 7 tables of a word a request, the chunks' masks and counts
    static_assert(kOffBar - kOffK >= (7 * kMaxBatch + 8 + kMaxBatch / 32 * 2) * 4, "plan");
};

// A stage of a ring, and how often it has been gone round (0 or 1)
struct Turn {
    int st = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++st == stages) st = 0, ph ^= 1;
    }
};

struct Params {
    int batch, q_rows, window, n_kv_heads, group, rt;
    int sms[kGroupSteps];  // CTAs that work where 2^i groups, or more, share a prefix
    int n_rows, slots_per_seq, block_size, max_blocks, num_pages, cap, prefix_cap;
    int box_rows;  // keys of a TMA box; 0: rows are gathered
    int map_rows;  // extent of the maps' second dimension
    uint32_t page_mul;
    int page_shift;
    bool paged, head_major;
    const int32_t *block_table, *seq_lens, *positions, *prefix_rows, *prefix_lens;
    const uint8_t *k, *v;
    const float *ks, *vs;
    int scale_shift;
    KvPlace place;
    float scale_log2;
    int4 *ws_rows;   // [batch * q_rows]: first row of ws_o for KV head 0, rows a part, parts
    // per row: log2 of the sum of weights (by what ws_o is held times), and of weights over scales
    float2 *ws_lse;
    uint16_t *ws_o;  // per row: HD f16
    int32_t *err;
};

// What a CTA works on.
struct Piece {
    int start, n_pos;  // the group's first position (b * q_rows) and its positions
    int prow, lo, hi;  // its prefix's row, the keys that some row of it may see
    int kt0, n_kt;     // key tiles
    int kvh, pair, split;
    int parts, base;   // parts of a row, first row of ws_o
};

// The keys [lo, hi) of its prefix that some row of request b attends.
__device__ __forceinline__ void request_range(const Params &p, int b, bool report, int &row,
                                              int &plen, int &lo, int &hi) {
    int len = p.seq_lens[b];
    plen = p.prefix_lens[b];
    row = p.prefix_rows[b];
    bool odd = len < 0 || len > p.cap || plen < 0 || plen > p.prefix_cap;
    len = max(0, min(len, p.cap));
    plen = max(0, min(plen, p.prefix_cap));
    int pmax = -1, oldest = INT32_MAX;
    for (int r = 0; r < p.q_rows; ++r) {
        const int pos = p.positions[(int64_t)b * p.q_rows + r];
        pmax = max(pmax, pos);
        if (pos >= 0) oldest = min(oldest, pos);
    }
    if (plen == 0) row = -1;
    const bool absent = plen > 0 && (row < 0 || row >= p.n_rows);
    if (report && (odd || absent)) report_error(p.err, ATTN_ERR_BOUNDS);
    hi = absent ? 0 : (int)min((int64_t)min(len, plen), (int64_t)pmax + 1);
    lo = p.window > 0 ? max(0, oldest - p.window + 1) : 0;
    if (hi <= lo) hi = 0, lo = INT32_MAX;
}

// How many groups share a prefix (the plan's count, from nothing but lengths and rows).
__device__ __forceinline__ int sharing_groups(const Params &p) {
    int n = 0;
    for (int b0 = 0; b0 < p.batch; b0 += blockDim.x) {
        const int b = b0 + (int)threadIdx.x;
        bool first = false;
        if (b < p.batch) {
            const int plen = max(0, min(p.prefix_lens[b], p.prefix_cap));
            first = plen > 0 && (b == 0 || p.prefix_rows[b] != p.prefix_rows[b - 1] ||
                                 plen != max(0, min(p.prefix_lens[b - 1], p.prefix_cap)));
        }
        n += __syncthreads_count(first);
    }
    return n;
}
__device__ __forceinline__ int working_ctas(const Params &p, int groups) {
    return p.sms[31 - __clz(max(1, groups))];
}

// The plan: groups, their pieces, and the piece that is asked for (n_kt 0: none).  `mem` is
// scratch in shared memory; every thread of the CTA calls this and passes its last barrier.  ctas:
// how many CTAs work (sharing_groups has to agree: a CTA that left by it takes no piece).  Of U units
// (group, KV head, pair of tiles) that weigh their key tiles each is cut into so many pieces (else
// 1 + floor((CTAs - U) tiles / sum)) that all are at most the CTAs, or U.
__device__ int make_plan(const Params &p, int32_t *mem, int want, bool tables, Piece &mine,
                         int &ctas) {
    const int kThreads = blockDim.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int B = p.batch, chunks = (B + 31) / 32;
    int32_t *r_lo = mem, *r_hi = r_lo + kMaxBatch, *g_start = r_hi + kMaxBatch;
    int32_t *g_lo = g_start + kMaxBatch + 8, *g_hi = g_lo + kMaxBatch, *g_parts = g_hi + kMaxBatch;
    int32_t *g_base = g_parts + kMaxBatch, *c_mask = g_base + kMaxBatch;
    int32_t *c_base = c_mask + kMaxBatch / 32;
    __shared__ int s_groups, s_total, s_ctas;
    for (int c = warp; c < chunks; c += kThreads / 32) {
        const int b = c * 32 + lane;
        bool first = false;
        int before_plen = 0, before_row = 0, row = 0, plen = 0;
        if (b < B) {
            int lo, hi;
            request_range(p, b, blockIdx.x == 0 && tables, row, plen, lo, hi);
            r_lo[b] = lo, r_hi[b] = hi;
            g_lo[b] = INT32_MAX, g_hi[b] = 0;
            before_plen = plen, before_row = row;
        }
        // the neighbour before: its length and row (-1 where it has no prefix)
        before_plen = __shfl_up_sync(0xffffffffu, before_plen, 1);
        before_row = __shfl_up_sync(0xffffffffu, before_row, 1);
        if (b < B) {
            if (lane == 0 && b > 0) {
                before_plen = max(0, min(p.prefix_lens[b - 1], p.prefix_cap));
                before_row = before_plen > 0 ? p.prefix_rows[b - 1] : -1;
            }
            first = b == 0 || before_plen != plen || before_row != row;
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, first);
        const uint32_t sharing = __ballot_sync(0xffffffffu, first && plen > 0);
        if (lane == 0) c_mask[c] = (int32_t)mask, c_base[c] = __popc(sharing);
    }
    if (threadIdx.x == 0) mine.n_kt = 0;
    __syncthreads();
    if (warp == 0) {
        int carry = 0, sharing = 0;
        for (int c0 = 0; c0 < chunks; c0 += 32) {
            const int n = c0 + lane < chunks ? __popc((uint32_t)c_mask[c0 + lane]) : 0;
            if (c0 + lane < chunks) sharing += c_base[c0 + lane];
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (c0 + lane < chunks) c_base[c0 + lane] = carry + x - n;
            carry += __shfl_sync(0xffffffffu, x, 31);
        }
        sharing = __reduce_add_sync(0xffffffffu, sharing);
        if (lane == 0) {
            s_groups = carry;
            g_start[carry] = B;
            s_ctas = working_ctas(p, sharing);
        }
    }
    __syncthreads();
    ctas = s_ctas;
    auto group_of = [&](int b) {
        const uint32_t upto = 0xffffffffu >> (31 - (b & 31));
        return c_base[b >> 5] + __popc((uint32_t)c_mask[b >> 5] & upto) - 1;
    };
    for (int b = threadIdx.x; b < B; b += kThreads) {
        const int g = group_of(b);
        if ((uint32_t)c_mask[b >> 5] >> (b & 31) & 1u) g_start[g] = b;
        if (r_hi[b] > 0) {
            atomicMin(&g_lo[g], r_lo[b]);
            atomicMax(&g_hi[g], r_hi[b]);
        }
    }
    __syncthreads();
    if (warp == 0) {
        const int groups = s_groups;
        auto tiles_of = [&](int g) {
            return g_hi[g] > 0 ? (g_hi[g] + kBN - 1) / kBN - g_lo[g] / kBN : 0;
        };
        auto pairs_of = [&](int g) {
            return ((g_start[g + 1] - g_start[g]) * p.q_rows + 2 * p.rt - 1) / (2 * p.rt);
        };
        int64_t work = 0;
        int units = 0;
        for (int g = lane; g < groups; g += 32) {
            const int t = tiles_of(g), u = t > 0 ? pairs_of(g) * p.n_kv_heads : 0;
            units += u;
            work += (int64_t)u * t;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            units += __shfl_xor_sync(0xffffffffu, units, o);
            work += __shfl_xor_sync(0xffffffffu, work, o);
        }
        // Of U units, each cut into pieces of at most s key tiles: the least s whose pieces are no
        // more than the CTAs lies between work / CTAs and work / (CTAs - U); 32 of those are tried
        const int spare = max(0, ctas - units);
        int most = 0;  // s, or 0: units are cut in proportion
        if (groups <= 32 && spare > 0 && work < (int64_t(1) << 30) && work > 0) {
            const int t = lane < groups ? tiles_of(lane) : 0;
            const int u = t > 0 ? pairs_of(lane) * p.n_kv_heads : 0;
            const int s0 = ((int)work + ctas - 1) / ctas, s1 = ((int)work + spare - 1) / spare;
            const int s = s0 + (int)(((int64_t)(s1 - s0) * lane + 30) / 31);
            int n = 0;
            for (int g = 0; g < groups; ++g) {
                const int tg = __shfl_sync(0xffffffffu, t, g), ug = __shfl_sync(0xffffffffu, u, g);
                n += ug * ((tg + s - 1) / s);
            }
            const uint32_t fits = __ballot_sync(0xffffffffu, n <= ctas);
            most = fits != 0 ? __shfl_sync(0xffffffffu, s, __ffs(fits) - 1) : 0;
        }
        int at = 0, row = 0;  // pieces and rows of ws_o before these groups
        for (int g0 = 0; g0 < groups; g0 += 32) {
            const int g = g0 + lane;
            int n = 0, rows = 0, cut = 0, pairs = 0, tiles = 0, n_pos = 0;
            bool two = false;
            if (g < groups) tiles = tiles_of(g);
            if (tiles > 0) {
                n_pos = (g_start[g + 1] - g_start[g]) * p.q_rows;
                pairs = pairs_of(g);
                cut = most > 0 ? (tiles + most - 1) / most
                               : min(tiles, 1 + (int)((int64_t)spare * tiles / work));
                n = pairs * p.n_kv_heads * cut;
                two = n_pos <= p.rt;  // one tile: two parts a piece
                rows = (two ? 2 : 1) * cut * p.n_kv_heads * n_pos * p.group;
            }
            int x = n, y = rows;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) x += a, y += b;
            }
            const int before = at + x - n, base = row + y - rows;
            if (g < groups) {
                g_parts[g] = (two ? 2 : 1) * cut;
                g_base[g] = base;
            }
            if (want >= before && want < before + n) {
                const int i = want - before, unit = i / cut;
                Piece m;
                m.start = g_start[g] * p.q_rows;
                m.n_pos = n_pos;
                m.prow = p.prefix_rows[g_start[g]];
                m.lo = g_lo[g], m.hi = g_hi[g];
                m.split = i - unit * cut;
                const int whole = tiles / cut, rest = tiles - whole * cut;
                m.kt0 = m.lo / kBN + m.split * whole + min(m.split, rest);
                m.n_kt = whole + (m.split < rest ? 1 : 0);
                m.kvh = unit / pairs;
                m.pair = unit - m.kvh * pairs;
                m.parts = (two ? 2 : 1) * cut;
                m.base = base;
                mine = m;
            }
            at += __shfl_sync(0xffffffffu, x, 31);
            row += __shfl_sync(0xffffffffu, y, 31);
        }
        if (lane == 0) s_total = at;
    }
    __syncthreads();
    // where the merge finds a position's parts
    if (tables && (int)blockIdx.x < ctas)
        for (int i = blockIdx.x * kThreads + threadIdx.x; i < B * p.q_rows; i += ctas * kThreads) {
            const int b = i / p.q_rows, g = group_of(b), n = g_start[g + 1] - g_start[g];
            p.ws_rows[i] = make_int4(g_base[g] + (i - g_start[g] * p.q_rows) * p.group,
                                     n * p.q_rows * p.group, g_parts[g], 0);
        }
    return s_total;
}

// Four codes -> two f16x2 words; exact.  INT8: a byte with its sign bit flipped is c + 128;
// behind the byte 0x64 it is the f16 1024 + (c + 128).
template <int FMT>
__device__ __forceinline__ void codes_to_f16(uint32_t x, uint32_t &lo, uint32_t &hi) {
    if constexpr (FMT == kE4M3) {
        lo = e4m3x2_to_f16x2(x);
        hi = e4m3x2_to_f16x2(x >> 16);
    } else {
        x ^= 0x80808080u;
        const uint32_t bias = 0x64806480u;  // 1152, twice
        lo = __byte_perm(x, 0x64646464u, 0x4140u);
        hi = __byte_perm(x, 0x64646464u, 0x4342u);
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(bias));
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(bias));
    }
}

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

__device__ __forceinline__ void mbar_inval(uint64_t *bar) {
    asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
}

// Instructions of one thread, chosen by `on`, in code that the whole warp runs: addresses and
// descriptors stay in uniform registers (behind `if (lane == 0)` every product first moves six
// words there, 75 cycles a product against the 64 that it takes).
__device__ __forceinline__ bool elect_one() {
    uint32_t on;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(on));
    return on != 0;
}
__device__ __forceinline__ void mma_ss_if(bool on, uint32_t d, uint64_t a, uint64_t b,
                                          uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"((uint32_t)on)
        : "memory");
}
__device__ __forceinline__ void mma_ts_if(bool on, uint32_t d, uint32_t a, uint64_t b,
                                          uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"((uint32_t)on)
        : "memory");
}
__device__ __forceinline__ void commit_if(bool on, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            smem_u32(bar)),
        "r"((uint32_t)on)
        : "memory");
}

// f16 words whose exponent is all ones become 0 in each half.
__device__ __forceinline__ uint32_t drop_nan(uint32_t w) {
    if ((w & 0x7C00u) == 0x7C00u) w &= 0xFFFF0000u;
    if ((w & 0x7C000000u) == 0x7C000000u) w &= 0x0000FFFFu;
    return w;
}

// bf16 NaN become 0 in each half.
__device__ __forceinline__ uint32_t drop_bf16_nan(uint32_t w) {
    if ((w & 0x7FFFu) > 0x7F80u) w &= 0xFFFF0000u;
    if ((w & 0x7FFF0000u) > 0x7F800000u) w &= 0x0000FFFFu;
    return w;
}

template <int FMT, int HD>
__global__ void __launch_bounds__(Cfg<FMT, HD>::kThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const Params p) {
    using C = Cfg<FMT, HD>;
    constexpr int kThreads = C::kThreads, kConv = C::kConv;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem, *sK = smem + C::kOffK, *sQ1 = smem + C::kOffQ1, *sV = smem + C::kOffV;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *k_full = bars;                  // [kMaxK] loaded (bf16)
    uint64_t *k_empty = k_full + C::kMaxK;    // [kMaxK] multiplied
    uint64_t *k_conv = k_empty + C::kMaxK;    // [kMaxK] ready, where the conversion passes it on
    uint64_t *v_full = k_conv + C::kMaxK;     // [kVStages]
    uint64_t *v_empty = v_full + C::kVStages;
    uint64_t *v_conv = v_empty + C::kVStages;
    uint64_t *raw_full = v_conv + C::kVStages;   // [kMaxRaw] codes
    uint64_t *raw_empty = raw_full + C::kMaxRaw;
    uint64_t *q_full = raw_empty + C::kMaxRaw;
    uint64_t *q_conv = q_full + 1;
    uint64_t *s_full = q_conv + 1;  // [2]
    uint64_t *p_full = s_full + 2;  // [2 tiles][2 key halves]
    uint64_t *o_done = p_full + 4;
    uint64_t *mma_done = o_done + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::kNumBars);
    __shared__ int s_bad;  // a page of the piece's keys is not in the pool
    __shared__ Piece w;    // (its fields are read where they are used: registers are short)
    // bf16: log2 of what a stage of V is multiplied with, and that
    __shared__ float2 s_by[C::kVStages];
    __shared__ uint32_t s_top[2][kConv / 32];  // ... largest magnitudes, by warp

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.group, R = p.q_rows, used = p.rt * G;
    const bool gather = p.box_rows == 0;

    if ((int)blockIdx.x >= p.sms[0]) {
        // at work only if there are more groups than one: out of the own keys' way else (with the
        // whole plan first 64 requests over 4,096 keys took 49.6 us)
        pdl_wait();
        pdl_launch_dependents();
        if ((int)blockIdx.x >= working_ctas(p, sharing_groups(p))) return;
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        prefetch_tensormap(&tm_q);
        if (!gather) {
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
        }
    }
    // Everything below may come from the previous kernel.  The own keys' launch begins behind this
    // wait of every CTA, so it reads what that one left without a wait of its own.
    pdl_wait();
    pdl_launch_dependents();

    int total = INT32_MAX, ctas = 1;
    for (int want = blockIdx.x; want < total; want += ctas) {
    if (threadIdx.x == 0) {
        for (int i = 0; want != (int)blockIdx.x && i < C::kNumBars; ++i) mbar_inval(&bars[i]);
        const int loads = gather ? 32 : 1;
        for (int s = 0; s < C::kMaxK; ++s) {
            mbar_init(&k_full[s], loads);
            mbar_init(&k_empty[s], 1);
            mbar_init(&k_conv[s], kConv);
        }
        for (int s = 0; s < C::kVStages; ++s) {
            mbar_init(&v_full[s], loads);
            mbar_init(&v_empty[s], 1);
            mbar_init(&v_conv[s], kConv);
        }
        for (int s = 0; s < C::kMaxRaw; ++s) {
            mbar_init(&raw_full[s], loads);
            mbar_init(&raw_empty[s], kConv);
        }
        mbar_init(q_full, 1);
        mbar_init(q_conv, 256);
        mbar_init(&s_full[0], 1);
        mbar_init(&s_full[1], 1);
        for (int i = 0; i < 4; ++i) mbar_init(&p_full[i], 128);
        mbar_init(o_done, 1);
        mbar_init(mma_done, 1);
        fence_barrier_init();
        s_bad = 0;
    }
    total = make_plan(p, reinterpret_cast<int32_t *>(sK), want, want == (int)blockIdx.x, w,
                      ctas);
    // Tile rows past the packed queries are never loaded: zeros
    if (used < kBM)
        for (int i = threadIdx.x; i < 2 * C::kHalves * (kBM - used) * 8; i += kThreads) {
            const int piece = i & 7, row = used + (i >> 3) % (kBM - used);
            const int th = (i >> 3) / (kBM - used);  // tile * halves + half
            *reinterpret_cast<uint4 *>((th < C::kHalves ? sQ : sQ1) + th % C::kHalves * (kBM * 128) +
                                       row * 128 + piece * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
    fence_proxy_async_smem();  // the plan's words and the zeros in Q, before copies and products
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // (the same for the whole CTA; it may lie past those that work, which for two groups can be
    // fewer than for one: its piece is then another's second one)
    if (w.n_kt == 0 || (int)blockIdx.x >= ctas) break;
    const uint32_t tmem = *tmem_slot;
    const int first_pos = w.pair * 2 * p.rt;         // of the group's positions
    const bool dual = w.n_pos <= p.rt;               // one tile, two streams of key tiles
    const int n_tiles = w.n_pos - first_pos > p.rt ? 2 : 1;
    const int k_stages = C::kKStages * C::kKSplit + (!C::kCodes && dual ? 1 : 0);  // of parts
    const int raw_stages = C::kRawStages + (C::kCodes && dual ? 2 : 0);
    uint8_t *sRaw = smem + C::kOffRaw - (dual ? C::kQBytes : 0);
    const int32_t *table = p.paged ? p.block_table + (int64_t)w.prow * p.max_blocks : nullptr;
    // t / block_size = t m / 2^(31 + L) for 0 <= t < 2^31, m = floor(2^(31 + L) / block_size) + 1,
    // 2^L >= block_size: m is less than 1 / block_size too large in the product
    auto block_of = [&](int t) { return (int)(((uint64_t)t * p.page_mul) >> p.page_shift); };
    auto page_of = [&](int t) { return __ldg(table + block_of(t)); };

    if (warp < kThreads / 32 - 8) {
        if (warp == 0 || warp == 2) {
            // ------------------------------------------------------------ loads
            const bool is_v = warp == 2;
            if (!is_v && lane == 0) {
                mbar_arrive_expect_tx(q_full, n_tiles * C::kHalves * used * 128);
                for (int a = 0; a < n_tiles; ++a)
                    for (int hf = 0; hf < C::kHalves; ++hf)
                        tma_load_3d((a == 0 ? sQ : sQ1) + hf * (kBM * 128), &tm_q, hf * 64,
                                    w.kvh * G, w.start + first_pos + a * p.rt, q_full);
            }
            __syncwarp();
            constexpr int kBytes = FMT == kBF16 ? C::kTileBytes : C::kRawBytes;
            const int n_kt = w.n_kt, kt0 = w.kt0, lo = w.lo, hi = w.hi, prow = w.prow, kvh = w.kvh;
            // this lane's box of a tile: whether it holds keys, its page, where it lies
            const int box0 = lane * p.box_rows;
            const bool boxed = !gather && box0 < kBN;
            const int x0 = p.head_major ? 0 : kvh * HD;
            auto holds = [&](int j) {
                const int t = (kt0 + j) * kBN + box0;
                return boxed && j < n_kt && t < hi && t + p.box_rows > lo;
            };
            auto read_page = [&](int j) {
                return p.paged && holds(j) ? page_of((kt0 + j) * kBN + box0) : 0;
            };
            auto place = [&](int j, int page) {
                const int t = (kt0 + j) * kBN + box0;
                if (!holds(j) || (p.paged && (unsigned)page >= (unsigned)p.num_pages))
                    return make_int2(p.map_rows, 0);  // outside the tensor: zeros
                // slot-major: slot y; head-major: row y of (block, head) z
                if (p.paged) {
                    const int r = t - block_of(t) * p.block_size;
                    return p.head_major ? make_int2(r, page * p.n_kv_heads + kvh)
                                        : make_int2(page * p.block_size + r, 0);
                }
                return p.head_major ? make_int2(t, prow * p.n_kv_heads + kvh)
                                    : make_int2(prow * p.slots_per_seq + t, 0);
            };
            auto send = [&](const CUtensorMap *map, int2 at, uint8_t *dst, uint64_t *bar) {
                if (lane == 0) mbar_arrive_expect_tx(bar, kBytes);
                __syncwarp();
                if (boxed) {
                    if constexpr (FMT == kBF16) {
                        for (int hf = 0; hf < C::kHalves; ++hf)
                            tma_load_3d(dst + hf * (kBN * 128) + box0 * 128, map, x0 + hf * 64, at.x,
                                        at.y, bar);
                    } else {
                        tma_load_3d(dst + box0 * HD, map, x0, at.x, at.y, bar);
                    }
                }
                __syncwarp();
            };
            // row by row: lane l finds rows l, l + 32, l + 64 and l + 96
            auto gather_rows = [&](const uint8_t *src, int j, uint8_t *dst, uint64_t *bar) {
                constexpr int kPieces = kBytes / kBN / 16;  // of a row
                const uint32_t to = smem_u32(dst);
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    const int t = (kt0 + j) * kBN + i * 32 + lane;
                    int64_t off = -1;
                    if (t < hi && t >= lo) {
                        const int page = page_of(t);
                        if ((unsigned)page < (unsigned)p.num_pages)
                            off = p.place.head_offset(
                                (int64_t)page * p.block_size + (t - block_of(t) * p.block_size), kvh);
                    }
#pragma unroll 4
                    for (int n = 0; n < kPieces; ++n) {
                        const int rr = n * (32 / kPieces) + lane / kPieces, piece = lane % kPieces;
                        const int64_t at = __shfl_sync(0xffffffffu, off, rr);
                        const int r = i * 32 + rr;
                        copy16(to + (piece >> 3) * (kBN * 128) + r * 128 +
                                   (((piece & 7) ^ (r & 7)) << 4),
                               src + (at < 0 ? 0 : at + piece * 16), at >= 0);
                    }
                }
                cp_async_arrive_noinc(bar);
            };
            // a tile's pages are read a tile before they are wanted; the ring of codes holds K and
            // V in turn
            uint64_t *empty = C::kCodes ? raw_empty : is_v ? v_empty : k_empty;
            uint64_t *full = C::kCodes ? raw_full : is_v ? v_full : k_full;
            uint8_t *ring = C::kCodes ? sRaw : is_v ? sV : sK;
            const CUtensorMap *map = is_v ? &tm_v : &tm_k;
            const int stages = C::kCodes ? raw_stages : is_v ? C::kVStages : k_stages;
            Turn t;
            if (C::kCodes && is_v) t.next(stages);
            int j = 0, page = read_page(0);
            for (; j < n_kt; ++j) {
                const int2 at = place(j, page);
                page = read_page(j + 1);
                const bool ok = mbar_wait(&empty[t.st], t.ph ^ 1, p.err);
                if (!__all_sync(0xffffffffu, ok)) break;
                if (gather)
                    gather_rows(is_v ? p.v : p.k, j, ring + t.st * kBytes, &full[t.st]);
                else
                    send(map, at, ring + t.st * kBytes, &full[t.st]);
                t.next(stages);
                if (C::kCodes) t.next(stages);
            }
            // No copy may still be landing when the CTA exits (normally all have been read)
            const int every = C::kCodes ? 2 : 1, first = C::kCodes && is_v ? 1 : 0;
            for (int i = max(0, j - stages / every); i < j; ++i) {
                const int n = i * every + first;
                mbar_wait(&full[n % stages], (n / stages) & 1, p.err);
            }
            if (!is_v) mbar_wait(q_full, 0, p.err);
        } else if (warp == 1) {
            // ------------------------------------------------------------ products
            {
                const bool on = elect_one();
                constexpr uint32_t idesc_qk = FMT == kBF16 ? idesc_bf16_f32(kBM, kBN, 0, 0)
                                                           : idesc_f16_f32(kBM, kBN, 0, 0);
                constexpr uint32_t idesc_pv = idesc_f16_f32(kBM, HD, 0, 1);
                const uint64_t q_desc = smem_desc_sw128(smem_u32(sQ), 16, 1024);
                const uint64_t k_desc0 = smem_desc_sw128(smem_u32(sK), 16, 1024);
                const uint64_t v_desc0 = smem_desc_sw128(smem_u32(sV), kBN * 128, 1024);
                Turn kt, vt;
                uint64_t *k_in = C::kCodes || gather ? k_conv : k_full;
                // Scores of Q tile qt into S a, when their K is there (wait: it may not be); done:
                // the tile of K is not wanted again
                auto issue_qk = [&](int a, int qt, bool wait, bool done) {
                    const uint64_t qd = q_desc + (uint64_t)((qt * C::kOffQ1) >> 4);
                    Turn t = kt;
#pragma unroll
                    for (int part = 0; part < C::kKSplit; ++part) {
                        if (wait && !mbar_wait(&k_in[t.st], t.ph, p.err)) return false;
                        tc_fence_after();
                        const uint64_t kd = k_desc0 + (uint64_t)((t.st * C::kKPart) >> 4);
                        constexpr int kSteps = HD / 16 / C::kKSplit;
#pragma unroll
                        for (int k = 0; k < kSteps; ++k) {
                            const int kk = part * kSteps + k;
                            mma_ss_if(on, tmem + a * 128,
                                      qd + (uint64_t)(((kk >> 2) * (kBM * 128) + (kk & 3) * 32) >> 4),
                                      kd + (uint64_t)(((k >> 2) * (kBN * 128) + (k & 3) * 32) >> 4),
                                      idesc_qk, kk > 0 ? 1u : 0u);
                        }
                        if (done) commit_if(on, &k_empty[t.st]);
                        t.next(k_stages);
                    }
                    commit_if(on, &s_full[a]);
                    if (done) kt = t;
                    return true;
                };
                auto issue_pv_half = [&](int a, int vst, int hh, bool first) {
                    const uint64_t vd = v_desc0 + (uint64_t)((vst * C::kTileBytes) >> 4);
                    const uint32_t p_tmem = tmem + a * 128;
                    const uint32_t o_tmem = tmem + 256 + a * HD;
#pragma unroll
                    for (int k4 = 0; k4 < kBN / 32; ++k4) {
                        const int kk = hh * (kBN / 32) + k4;
                        mma_ts_if(on, o_tmem, p_tmem + kk * 8,
                                  vd + (uint64_t)((kk * 16 * 128) >> 4), idesc_pv,
                                  (!first || k4 > 0) ? 1u : 0u);
                    }
                };
                // the weights of a stream's jj-th key tile into its output
                auto pv = [&](int a, int jj) {
                    for (int hh = 0; hh < 2; ++hh) {
                        if (!mbar_wait(&p_full[a * 2 + hh], jj & 1, p.err)) return false;
                        tc_fence_after();
                        issue_pv_half(a, vt.st, hh, jj == 0 && hh == 0);
                    }
                    return true;
                };
                const int n_kt = w.n_kt;
                bool ok = mbar_wait(FMT == kBF16 ? q_full : q_conv, 0, p.err);
                if (dual) {
                    // tile j belongs to stream j & 1
                    for (int j = 0; ok && j < min(2, n_kt); ++j) ok = issue_qk(j, 0, true, true);
                    for (int j = 0; ok && j < n_kt; ++j) {
                        ok = mbar_wait(&v_conv[vt.st], vt.ph, p.err) && pv(j & 1, j >> 1);
                        if (!ok) break;
                        commit_if(on, &v_empty[vt.st]);
                        vt.next(C::kVStages);
                        if (j + 2 < n_kt) ok = issue_qk(j & 1, 0, true, true);
                    }
                } else {
                    for (int a = 0; ok && a < n_tiles; ++a)
                        ok = issue_qk(a, a, a == 0, a == n_tiles - 1);
                    for (int j = 0; ok && j < n_kt; ++j) {
                        ok = mbar_wait(&v_conv[vt.st], vt.ph, p.err);
                        for (int a = 0; ok && a < n_tiles; ++a) {
                            ok = pv(a, j);
                            if (!ok) break;
                            if (a == n_tiles - 1) commit_if(on, &v_empty[vt.st]);
                            if (j + 1 < n_kt) ok = issue_qk(a, a, a == 0, a == n_tiles - 1);
                        }
                        vt.next(C::kVStages);
                    }
                }
                commit_if(on, o_done);
                commit_if(on, mma_done);
                mbar_wait(mma_done, 0, p.err);
            }
        } else if (warp >= 4) {
            // ------------------------------------------------------------ into f16
            const int ct = threadIdx.x & (kConv - 1);
            // keys of a tile that lie in the group's range
            auto inside = [&](int tile, int row) {
                const int t = tile * kBN + row;
                return t >= w.lo && t < w.hi;
            };
            auto whole = [&](int tile) {
                return tile * kBN >= w.lo && tile * kBN + kBN <= w.hi;
            };
            // The largest of the four warps' values (two tables in turn: one is written again behind
            // the next barrier)
            int table_at = 0;
            auto largest = [&](__nv_bfloat162 most) {
                const uint32_t two = *reinterpret_cast<const uint32_t *>(&most);
                const uint32_t mine = __reduce_max_sync(0xffffffffu, max(two >> 16, two & 0xFFFFu));
                uint32_t *to = s_top[table_at];
                table_at ^= 1;
                if (lane == 0) to[ct >> 5] = mine;
                asm volatile("bar.sync 4, %0;" ::"n"(kConv) : "memory");
                uint32_t top = to[0];
#pragma unroll
                for (int i = 1; i < kConv / 32; ++i) top = max(top, to[i]);
                return top;
            };
            const __nv_bfloat162 zero2 = __bfloat162bfloat162(__ushort_as_bfloat16(0));
            auto size_of = [](__nv_bfloat162 most, uint32_t u) {
                return __hmax2_nan(most, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&u)));
            };
            auto power = [](int shift) {
                return __bfloat162bfloat162(
                    __ushort_as_bfloat16((unsigned short)((127 + shift) << 7)));
            };
            auto to_f16 = [](uint32_t u, __nv_bfloat162 by) {
                const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&u), by);
                return bf16x2_to_f16x2_sat(*reinterpret_cast<const uint32_t *>(&y));
            };
            // A tile of bf16 V in place, to f16 times 2^shift; returns the largest |x| of its keys in
            // the group's range, as a bf16 pattern
            auto v_in_place = [&](int tile, uint32_t at, int shift) {
                const bool all = whole(tile);
                constexpr int kBatch = 4;  // pieces read before one is written (eight: 1% slower)
                __nv_bfloat162 most = zero2;
                const __nv_bfloat162 by = power(shift);
#pragma unroll 1
                for (int i0 = ct; i0 < C::kTileBytes / 16; i0 += kConv * kBatch) {
                    uint4 x[kBatch];
#pragma unroll
                    for (int b = 0; b < kBatch; ++b)
                        x[b] = ld_shared_v4(at + (i0 + kConv * b) * 16);
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {
                        const int i = i0 + kConv * b;
                        if (!all && !inside(tile, (i >> 3) & (kBN - 1)))
                            x[b] = make_uint4(0u, 0u, 0u, 0u);
                        uint32_t *u = &x[b].x;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            most = size_of(most, u[e]);
                            u[e] = to_f16(u[e], by);
                        }
                        st_shared_v4(at + i * 16, x[b]);
                    }
                }
                return largest(most);
            };
            // The power of two that brings a largest value to 2^9 .. 2^10: tiles of 2^-13 to 2^5 times
            // its size do by it
            auto shift_of = [](uint32_t top) {
                return min(max(136 - (int)(top >> 7), 0), kShiftTop);
            };
            // ... that a piece begins with: by a quarter of its first tile (a wrong guess costs what
            // v_again takes: two requests over 512 keys of 2^-10 27.2 us where 1 was tried first and the
            // tile read piece by piece, 16.9 so)
            auto first_guess = [&](int tile, uint32_t at) {
                __nv_bfloat162 most = zero2;
#pragma unroll
                for (int b = 0; b < C::kTileBytes / 16 / kConv / 4; ++b) {
                    const int i = ct + kConv * b * 4;
                    const uint4 x = ld_shared_v4(at + i * 16);
                    if (!inside(tile, (i >> 3) & (kBN - 1))) continue;
                    most = size_of(size_of(most, x.x), x.y);
                    most = size_of(size_of(most, x.z), x.w);
                }
                const uint32_t top = largest(most);
                return top == 0 ? 0 : shift_of(top);
            };
            // The same from the cache, where the power of two was not right for a largest value `top`
            // (a NaN, which is taken as 0: whatever the others' is); returns the shift taken
            auto v_again = [&](int tile, uint32_t at, uint32_t top) {
                auto piece = [&](int i) {  // piece i of the tile in shared memory (swizzled)
                    const int r = (i >> 3) & (kBN - 1), t = tile * kBN + r;
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if (!inside(tile, r)) return x;
                    int64_t slot = (int64_t)w.prow * p.slots_per_seq + t;
                    if (p.paged) {
                        const int page = page_of(t);
                        if ((unsigned)page >= (unsigned)p.num_pages) return x;
                        slot = (int64_t)page * p.block_size + (t - block_of(t) * p.block_size);
                    }
                    return __ldcg(reinterpret_cast<const uint4 *>(
                        p.v + p.place.head_offset(slot, w.kvh) + (i / (kBN * 8)) * 128 +
                        (((i ^ r) & 7) << 4)));
                };
                if (top > 0x7F80u) {
                    __nv_bfloat162 most = zero2;
#pragma unroll 1
                    for (int i = ct; i < C::kTileBytes / 16; i += kConv) {
                        const uint4 x = piece(i);
                        most = size_of(size_of(most, drop_bf16_nan(x.x)), drop_bf16_nan(x.y));
                        most = size_of(size_of(most, drop_bf16_nan(x.z)), drop_bf16_nan(x.w));
                    }
                    top = largest(most);
                }
                const int shift = shift_of(top);
                const __nv_bfloat162 by = power(shift);
#pragma unroll 1
                for (int i0 = ct; i0 < C::kTileBytes / 16; i0 += kConv * 4) {
                    uint4 x[4];
#pragma unroll
                    for (int b = 0; b < 4; ++b) x[b] = piece(i0 + kConv * b);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        uint32_t *u = &x[b].x;
#pragma unroll
                        for (int e = 0; e < 4; ++e) u[e] = to_f16(drop_bf16_nan(u[e]), by);
                        st_shared_v4(at + (i0 + kConv * b) * 16, x[b]);
                    }
                }
                return shift;
            };
            // 64 dims of a tile of codes (half hf) from `from` into f16 rows at `to`.  Eight lanes
            // read 4 pieces (16 codes) of rows r and r ^ 5 (128-byte rows, swizzled) or of two rows
            // (64-byte ones), so that neither their loads nor their stores (pieces 2 i and 2 i + 1
            // of f16 rows of 128 bytes, swizzled) meet in a bank.
            auto widen = [&](bool is_v, int tile, uint32_t from, int hf, uint32_t to) {
                const bool all = !is_v || whole(tile);
                constexpr int kRounds = kBN / 8 / (kConv / 32);  // of 8 rows a warp
                const int l = ct & 31, ph = l >> 3, second = (l >> 2) & 1, piece = l & 3;
                const int row0 = (ct >> 5) * 8 + (HD == 128 ? (second ? ph ^ 5 : ph) : 2 * ph + second);
                // rows row0, row0 + 32, ..: their swizzle is the same
                uint32_t src = HD == 128 ? from + row0 * 128 + (((hf * 4 + piece) ^ (row0 & 7)) << 4)
                                         : from + row0 * 64 + piece * 16;
                uint32_t dst0 = to + row0 * 128 + (((2 * piece) ^ (row0 & 7)) << 4);
                uint32_t dst1 = to + row0 * 128 + (((2 * piece + 1) ^ (row0 & 7)) << 4);
                // (rolled: eight pieces at once took as long, and with all warps' code long the
                // instruction cache is short)
                uint4 next = ld_shared_v4(src);
#pragma unroll 2
                for (int i = 0; i < kRounds; ++i) {
                    const uint4 x = next;
                    src += 32 * (HD == 128 ? 128 : 64);
                    if (i + 1 < kRounds) next = ld_shared_v4(src);
                    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
                    uint32_t h[8], odd = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) codes_to_f16<FMT>(u[e], h[2 * e], h[2 * e + 1]);
                    if (is_v) {
                        const bool on = all || inside(tile, row0 + 32 * i);
                        if (FMT == kE4M3) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) odd |= (u[e] & 0x7F7F7F7Fu) + 0x01010101u;
                            odd &= 0x80808080u;  // a code of NaN, 0x7F or 0xFF
                        }
                        if (odd != 0 || !on) {
                            if (on) report_error(p.err, ATTN_ERR_UNSUPPORTED);
#pragma unroll
                            for (int e = 0; e < 8; ++e) h[e] = on ? drop_nan(h[e]) : 0u;
                        }
                    }
                    st_shared_v4(dst0, make_uint4(h[0], h[1], h[2], h[3]));
                    st_shared_v4(dst1, make_uint4(h[4], h[5], h[6], h[7]));
                    dst0 += 32 * 128, dst1 += 32 * 128;
                }
            };
            Turn kt, vt, rt;
            bool ok = true;
            int shift = 0;  // log2 of what values are multiplied with
            if constexpr (C::kCodes) {
                const bool is_v = warp >= 8;
                const int stages = is_v ? C::kVStages : k_stages;
                uint64_t *empty = is_v ? v_empty : k_empty, *done = is_v ? v_conv : k_conv;
                const uint32_t ring = smem_u32(is_v ? sV : sK);
                if (is_v) rt.next(raw_stages);  // (the ring holds K and V in turn)
                for (int j = 0; ok && j < w.n_kt; ++j) {
                    ok = mbar_wait(&raw_full[rt.st], rt.ph, p.err);
                    // V by tiles, K by halves
#pragma unroll 1
                    for (int hf = 0; ok && hf < C::kHalves; ++hf) {
                        if (!is_v || hf == 0) ok = mbar_wait(&empty[vt.st], vt.ph ^ 1, p.err);
                        if (!ok) break;
                        const uint32_t at = is_v ? vt.st * C::kTileBytes + hf * (kBN * 128)
                                                 : vt.st * C::kKPart;
                        widen(is_v, w.kt0 + j, smem_u32(sRaw + rt.st * C::kRawBytes), hf, ring + at);
                        if (is_v && hf + 1 < C::kHalves) continue;
                        fence_proxy_async_smem();
                        mbar_arrive(&done[vt.st]);
                        vt.next(stages);
                    }
                    mbar_arrive(&raw_empty[rt.st]);
                    rt.next(raw_stages);
                    rt.next(raw_stages);
                }
            } else {
                // (no way out where a wait ran out: the four warps meet at a barrier)
                ok = mbar_wait(&v_full[0], 0, p.err);
                shift = first_guess(w.kt0, smem_u32(sV));
                for (int j = 0; j < w.n_kt; ++j) {
                    if (gather) {
                        // K copied by cp.async: written again, so that this thread's fence
                        // covers what the tensor cores read
                        const uint32_t at = smem_u32(sK + kt.st * C::kTileBytes);
                        if (ok) ok = mbar_wait(&k_full[kt.st], kt.ph, p.err);
#pragma unroll 4
                        for (int i = ct; i < C::kTileBytes / 16; i += kConv)
                            st_shared_v4(at + i * 16, ld_shared_v4(at + i * 16));
                        fence_proxy_async_smem();
                        mbar_arrive(&k_conv[kt.st]);
                        kt.next(k_stages);
                    }
                    if (ok) ok = mbar_wait(&v_full[vt.st], vt.ph, p.err);
                    const uint32_t at = smem_u32(sV + vt.st * C::kTileBytes);
                    const int tile = w.kt0 + j;
                    const uint32_t top = v_in_place(tile, at, shift);
                    // f16 holds 65504 at most, and of what is 2^-4 at least all that counts: a
                    // value below 2^-14 is off by 2^-21 of the largest at most
                    const int size = (int)(top >> 7) + shift - 127;
                    if (top >= 0x4780u || size > (shift == 0 ? 15 : 14) ||
                        (top != 0 && size < -4 && shift < kShiftTop)) {
                        if (top >= 0x4780u) report_error(p.err, ATTN_ERR_UNSUPPORTED);
                        shift = v_again(tile, at, top);
                    }
                    // (zeros weigh nothing beside any other tile)
                    if (ct == 0) {
                        const int of = top == 0 ? kShiftTop : shift;
                        s_by[vt.st] = make_float2((float)of, __int_as_float((127 + of) << 23));
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(&v_conv[vt.st]);
                    vt.next(C::kVStages);
                }
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax
        const int a = (warp >> 2) & 1 ^ (C::kCodes ? 1 : 0);  // which tile, or stream
        const int quad = warp & 3;         // TMEM lane quadrant of this warp
        const int row = quad * 32 + lane;  // tile row = TMEM lane
        const int st = threadIdx.x - (kThreads - 256);  // 0 .. 255
        // a page that is not there is reported, and its keys are looked for in every tile
        if (p.paged) {
            const int b0 = max(w.lo, w.kt0 * kBN) / p.block_size;
            // (the last key's page; no sum of an end and a page's size, which may pass 31 bits)
            const int b1 = (min(w.hi, (w.kt0 + w.n_kt) * kBN) - 1) / p.block_size + 1;
            bool bad = false;
            for (int i = b0 + st; i < b1; i += 256)
                bad |= (unsigned)__ldg(table + i) >= (unsigned)p.num_pages;
            if (bad) {
                s_bad = 1;
                report_error(p.err, ATTN_ERR_BOUNDS);
            }
        }
        if constexpr (FMT != kBF16) {
            // q to f16 in place
            if (mbar_wait(q_full, 0, p.err)) {
                uint32_t big = 0;
                for (int i = st; i < n_tiles * C::kQBytes / 16; i += 256) {
                    const int tile = i / (C::kQBytes / 16);
                    const uint32_t at = smem_u32(tile == 0 ? sQ : sQ1 - C::kQBytes);
                    uint4 x = ld_shared_v4(at + i * 16);
                    uint32_t *u = &x.x;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t h = bf16x2_to_f16x2(u[e]);
                        // overflowed, NaN aside (which stays one, in its row)
                        if ((h & 0x7FFFu) == 0x7C00u || (h & 0x7FFF0000u) == 0x7C000000u) big = 1;
                        u[e] = h;
                    }
                    st_shared_v4(at + i * 16, x);
                }
                if (big) report_error(p.err, ATTN_ERR_UNSUPPORTED);
            }
            fence_proxy_async_smem();
            mbar_arrive(q_conv);
        }
        asm volatile("bar.sync 3, 256;" ::: "memory");
        const bool any_bad = *reinterpret_cast<volatile int *>(&s_bad) != 0;

        const int tile_pos = first_pos + (dual ? 0 : a * p.rt);  // the tile's first position
        const int live_rows = min(used, (w.n_pos - tile_pos) * G);
        const bool live = row < live_rows;
        int qi = -1, key_cap = -1;  // the row's position, and the last shared key it may see
        if (live) {
            const int i = w.start + tile_pos + row / G, b = i / R;
            qi = max(p.positions[i], -1);  // (below zero: no keys)
            const int len = max(0, min(p.seq_lens[b], p.cap));
            key_cap = min(min(qi, len - 1), max(0, min(p.prefix_lens[b], p.prefix_cap)) - 1);
        }
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        const uint32_t s_tmem = tmem + a * 128 + lane_base;
        const uint32_t o_tmem = tmem + 256 + a * HD + lane_base;
        const float sl2 = p.scale_log2;
        float m_run = -INFINITY, l_run = 0.f, w_run = 0.f;
        bool ok = true;
        // this warpgroup's key tiles
        const int j0 = dual ? a : 0, step = dual ? 2 : 1;
        Turn vt;  // ... and their stages of V
        if (j0 > 0) vt.next(C::kVStages);
        const int mine = a < n_tiles || dual ? (w.n_kt - j0 + step - 1) / step : 0;
        // scales of the 16 keys 16 (lane % 8) .. of a tile, read a tile ahead
        float next_k = 1.f, next_v = 1.f;
        auto read_scales = [&](int j) {
            next_k = next_v = 1.f;
            const int t = (w.kt0 + j) * kBN + 16 * (lane & 7);
            if (p.ks == nullptr || j >= w.n_kt || t >= w.hi || t + 16 <= w.lo) return;
            int64_t slot;
            if (p.paged) {
                const int page = page_of(t);
                if ((unsigned)page >= (unsigned)p.num_pages) return;
                slot = (int64_t)page * p.block_size + (t - block_of(t) * p.block_size);
            } else {
                slot = (int64_t)w.prow * p.slots_per_seq + t;
            }
            const int64_t at = (slot >> p.scale_shift) * p.n_kv_heads + w.kvh;
            next_k = __ldg(p.ks + at);
            next_v = __ldg(p.vs + at);
        };
        if constexpr (FMT != kBF16) read_scales(j0);
        for (int jj = 0; jj < mine; ++jj) {
            const int j = j0 + jj * step;
            float f_lane = sl2, lv_lane = 0.f, inv_lane = 1.f;
            if constexpr (FMT != kBF16) {
                if (p.ks != nullptr) {
                    const float sv = fmaxf(next_v, kScaleFloor);
                    f_lane = fminf(fmaxf(fmaxf(next_k, kScaleFloor) * sl2, 0x1p-126f), kFactorTop);
                    lv_lane = fast_log2(sv);
                    inv_lane = 0.25f * fast_rcp(0.25f * sv);  // subnormal from 2^126 on, not 0
                }
                read_scales(j + step);
            }
            // bf16: log2 of what the tile's values were multiplied with, and that (the stage is not
            // converted again before this warpgroup's weights are there).  Where it is waited for
            // shows: pairs before S (256 requests over 32,768 keys 158 us, behind the maximum 166),
            // lone tiles behind the maximum (two requests 16.0 us, before S 16.7)
            float2 by = make_float2(0.f, 1.f);
            auto wait_v = [&] {
                if (!mbar_wait(&v_conv[vt.st], vt.ph, p.err)) return false;
                by = s_by[vt.st];
                vt.next(C::kVStages);
                if (dual) vt.next(C::kVStages);
                return true;
            };
            if (FMT == kBF16 && !dual) ok = wait_v();
            ok = __all_sync(0xffffffffu, ok && mbar_wait(&s_full[a], jj & 1, p.err));
            if (!ok) break;
            tc_fence_after();
            const int key0 = (w.kt0 + j) * kBN;
            // the row sees columns lo <= c <= hi (c = key - key0)
            const int hi = key_cap - key0, lo = p.window > 0 ? qi - p.window + 1 - key0 : 0;
            const bool masked = hi < kBN - 1 || lo > 0 || any_bad;
            // Scores of columns c0 .. c0 + 31, -inf where the row does not see the key, back in
            // TMEM too
            auto mask = [&](float(&s)[32], int c0) {
                uint32_t see = c0 > hi || c0 + 31 < lo ? 0u : 0xffffffffu;
                if (hi - c0 < 31) see &= (2u << max(0, hi - c0)) - 1u;
                if (lo > c0) see &= 0xffffffffu << min(31, lo - c0);
                if (any_bad) {
                    const int t = key0 + c0 + lane;
                    see &= ~__ballot_sync(0xffffffffu,
                                          t >= w.lo && t < w.hi &&
                                              (unsigned)page_of(t) >= (unsigned)p.num_pages);
                }
#pragma unroll
                for (int c = 0; c < 32; ++c) s[c] = see >> c & 1u ? s[c] : -INFINITY;
                tmem_st_32x32b_x32(s_tmem + c0, *reinterpret_cast<uint32_t(*)[32]>(s));
            };
            // S is read from TMEM twice, 64 columns at a time, and the loops are kept rolled:
            // all 128 in registers leave too few for the rest, and unrolled code waits for the
            // instruction cache (the two warpgroups run different parts of it)
            float s0[32], s1[32];
            uint32_t(&u0)[32] = *reinterpret_cast<uint32_t(*)[32]>(s0);
            uint32_t(&u1)[32] = *reinterpret_cast<uint32_t(*)[32]>(s1);
            float mx = -INFINITY;
            auto top = [&](const float(&s)[32], int c0) {
                if constexpr (FMT == kBF16) {
                    float m0 = s[0], m1 = s[1], m2 = s[2], m3 = s[3];
#pragma unroll
                    for (int c = 4; c + 8 <= 32; c += 8) {
                        m0 = max3(m0, s[c], s[c + 1]);
                        m1 = max3(m1, s[c + 2], s[c + 3]);
                        m2 = max3(m2, s[c + 4], s[c + 5]);
                        m3 = max3(m3, s[c + 6], s[c + 7]);
                    }
                    m0 = max3(m0, s[28], s[29]), m1 = max3(m1, s[30], s[31]);
                    mx = max3(mx, max3(m0, m1, m2), m3);
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        // x = s f + lv grows with s (f > 0): its maximum is that of s
                        const float *x = s + 16 * i;
                        float m0 = max3(x[0], x[1], x[2]), m1 = max3(x[3], x[4], x[5]);
                        m0 = max3(m0, x[6], x[7]), m1 = max3(m1, x[8], x[9]);
                        m0 = max3(m0, x[10], x[11]), m1 = max3(m1, x[12], x[13]);
                        mx = fmaxf(mx, fmaf(max3(m0, m1, fmaxf(x[14], x[15])),
                                            __shfl_sync(0xffffffffu, f_lane, c0 / 16 + i),
                                            __shfl_sync(0xffffffffu, lv_lane, c0 / 16 + i)));
                    }
                }
            };
            const bool any_masked = __any_sync(0xffffffffu, masked);
#pragma unroll 1
            for (int c0 = 0; c0 < kBN; c0 += 64) {
                tmem_ld_32x32b_x32(s_tmem + c0, u0);
                tmem_ld_32x32b_x32(s_tmem + c0 + 32, u1);
                tmem_wait_ld();
                tmem_regs_after_wait(u0);
                tmem_regs_after_wait(u1);
                if (any_masked) {
                    mask(s0, c0);
                    mask(s1, c0 + 32);
                    tmem_wait_st();
                }
                top(s0, c0);
                top(s1, c0 + 32);
            }
            if constexpr (FMT == kBF16) {
                if (dual) ok = __all_sync(0xffffffffu, wait_v());
                if (!ok) break;
                mx = fmaf(mx, sl2, -by.x);
            }
            tmem_ld_32x32b_x32(s_tmem, u0);  // (under way meanwhile)
            float alpha = 1.f;
            if (mx > m_run + kRescaleLog2 || m_run == -INFINITY) {
                const float m_new = mx == -INFINITY ? m_run : mx;
                alpha = m_run == -INFINITY ? 0.f : fast_exp2(m_run - m_new);
                m_run = m_new;
            }
            if (jj > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                for (int c0 = 0; c0 < HD; c0 += 32) {
                    tmem_ld_32x32b_x32(o_tmem + c0, u1);
                    tmem_wait_ld();
                    tmem_regs_after_wait(u1);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        u1[e] = __float_as_uint(__uint_as_float(u1[e]) * alpha);
                    tmem_st_32x32b_x32(o_tmem + c0, u1);
                }
            }
            const float m_w = (m_run == -INFINITY ? 0.f : m_run) - kWeightLog2;
            float sum = 0.f, over = 0.f;
            // weights of columns c0 .. c0 + 31: over their own S columns, 32 keys in 16
            auto weigh = [&](float(&s)[32], int c0) {
                uint32_t pk[16];
                float sum0 = 0.f, sum1 = 0.f, f = sl2, shift = -m_w - by.x;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (FMT != kBF16 && (e & 7) == 0) {
                        f = __shfl_sync(0xffffffffu, f_lane, c0 / 16 + e / 8);
                        shift = __shfl_sync(0xffffffffu, lv_lane, c0 / 16 + e / 8) - m_w;
                    }
                    float x0, x1;
                    fma2(x0, x1, s[2 * e], s[2 * e + 1], f, f, shift, shift);
                    const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                    add2(sum0, sum1, sum0, sum1, p0, p1);
                    pk[e] = pack_f16x2(p0, p1);
                    if (FMT != kBF16 && (e & 7) == 7) {  // the end of 16 keys
                        sum += sum0 + sum1;
                        over = fmaf(sum0 + sum1,
                                    __shfl_sync(0xffffffffu, inv_lane, c0 / 16 + e / 8), over);
                        sum0 = sum1 = 0.f;
                    }
                }
                if (FMT == kBF16) sum += sum0 + sum1;
                tmem_st_32x32b_x16(s_tmem + c0 / 2, pk);
            };
            // (P of 32 columns lies in front of the S that is still to be read)
#pragma unroll 1
            for (int c0 = 0; c0 < kBN; c0 += 64) {
                tmem_wait_ld();
                tmem_regs_after_wait(u0);
                tmem_ld_32x32b_x32(s_tmem + c0 + 32, u1);
                weigh(s0, c0);
                tmem_wait_ld();
                tmem_regs_after_wait(u1);
                if (c0 + 64 < kBN) tmem_ld_32x32b_x32(s_tmem + c0 + 64, u0);
                weigh(s1, c0 + 32);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&p_full[a * 2 + c0 / 64]);
            }
            l_run = l_run * alpha + (FMT == kBF16 ? sum * by.y : over);
            w_run = w_run * alpha + sum;
        }
        if (m_run != -INFINITY && !(fabsf(m_run) < kScoreTop))
            report_error(p.err, ATTN_ERR_UNSUPPORTED);
        // ---- the state of each row: O over the sum of its weights, and both sums
        if (ok) mbar_wait(o_done, 0, p.err);
        __syncwarp();
        tc_fence_after();
        const bool any = !(w_run == 0.f);  // a key was seen (or a NaN met)
        float norm = any ? 1.f / w_run : 0.f;
        const int part = dual ? 2 * w.split + a : w.split;
        const int64_t row0 = (int64_t)w.base +
                             ((int64_t)w.kvh * w.parts + part) * ((int64_t)w.n_pos * G) +
                             (int64_t)tile_pos * G;
        if (dual || a < n_tiles) {
            // Through shared memory (the K ring for a = 0, the V ring for a = 1: the last
            // product has read them) as swizzled 128-byte rows of 64 dims, and out in whole
            // lines: a row a thread would write into 32 lines an instruction
            uint8_t *stage = a == 0 ? sK : sV;
            uint32_t orow[32];
            auto read_o = [&](int c0) {
                if (mine > 0) {  // warpgroup-uniform: O was accumulated into
                    tmem_ld_32x32b_x32(o_tmem + c0, orow);
                    tmem_wait_ld();
                    tmem_regs_after_wait(orow);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) orow[e] = 0u;
                }
            };
            // The row's largest output to 2^12 .. 2^13 (f16 ends at 2^16)
            float most = 0.f;
#pragma unroll 1
            for (int c0 = 0; c0 < HD; c0 += 32) {
                read_o(c0);
#pragma unroll
                for (int e = 0; e < 32; ++e) most = fmaxf(most, fabsf(__uint_as_float(orow[e])));
            }
            const int held = most > 0.f && isfinite(most * norm)
                                 ? min(max(139 - (int)(__float_as_uint(most * norm) >> 23), -30), 40)
                                 : 0;
            norm *= __int_as_float((127 + held) << 23);
#pragma unroll 1
            for (int c0 = 0; c0 < HD; c0 += 32) {
                read_o(c0);
                auto v = [&](int e) { return any ? __uint_as_float(orow[e]) * norm : 0.f; };
                const uint32_t base = smem_u32(stage + (c0 / 64) * (kBM * 128) + row * 128);
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                    const int piece = ((c0 & 63) >> 3) + q4;
                    st_shared_v4(base + ((piece ^ (row & 7)) << 4),
                                 make_uint4(pack_f16x2(v(8 * q4), v(8 * q4 + 1)),
                                            pack_f16x2(v(8 * q4 + 2), v(8 * q4 + 3)),
                                            pack_f16x2(v(8 * q4 + 4), v(8 * q4 + 5)),
                                            pack_f16x2(v(8 * q4 + 6), v(8 * q4 + 7))));
                }
            }
            if (live) {
                const float at = (m_run == -INFINITY ? 0.f : m_run) - kWeightLog2;
                p.ws_lse[row0 + row] = any ? make_float2(at - (float)held + __log2f(w_run),
                                                         at + __log2f(l_run))
                                           : make_float2(-INFINITY, -INFINITY);
            }
            if (a == 0)
                asm volatile("bar.sync 1, 128;" ::: "memory");
            else
                asm volatile("bar.sync 2, 128;" ::: "memory");
            uint4 *dst = reinterpret_cast<uint4 *>(p.ws_o + row0 * HD);
            for (int i = row; i < live_rows * (HD / 8); i += 128) {
                const int r = i / (HD / 8), piece = i % (HD / 8);
                dst[i] = ld_shared_v4(smem_u32(stage + (piece >> 3) * (kBM * 128) + r * 128) +
                                      (((piece & 7) ^ (r & 7)) << 4));
            }
        }
    }
    __syncwarp();  // (lanes that elected ones of their warp went ahead of)
    if (want + ctas >= total) break;
    tc_fence_before();  // another piece: everything has been read
    __syncthreads();
    tc_fence_after();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(*tmem_slot, kTmemCols);
}

struct MergeParams {
    const int4 *ws_rows;
    const float2 *ws_lse;
    const uint16_t *ws_o;
    AttendParts own;  // of the keys behind the prefixes
    __nv_bfloat16 *out;
    int q_rows, rows, n_q_heads, n_kv_heads, group;
    int first_row, n_rows;  // the launch's rows of a KV head, over the whole batch
};

// A row of the output from its parts: those of the shared keys, then those of its own.
// SPLIT warps a row, each every SPLIT-th part, a lane HD / 32 dims; the sums of 32 parts come in one
// load, the parts' outputs then wait for nothing.  Bound by those two round trips behind the last
// of both launches (~3 us; 8.5 us cold for 2,048 rows of 128 dims, 5.8 MB read).
template <int HD, int SPLIT>
__global__ void __launch_bounds__(256, SPLIT == 1 ? 4 : 2) shared_merge_kernel(const MergeParams p) {
    constexpr int V = HD / 32, kRows = 8 / SPLIT;
    __shared__ float sm_acc[SPLIT > 1 ? 8 : 1][HD];
    __shared__ float sm_m[8], sm_sum[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const AttendParts &a = p.own;
    // rows (entry, row of its block, head of the group) of each KV head in turn
    const int64_t i = (int64_t)blockIdx.x * kRows + warp / SPLIT;
    const int kvh = (int)(i / p.n_rows), q = (int)(i - (int64_t)kvh * p.n_rows) + p.first_row;
    const int b = q / p.rows, q_row = q - b * p.rows, rb = q_row / a.rb, row = q_row - rb * a.rb;
    const bool live = kvh < p.n_kv_heads;
    const int r = q_row / p.group, gh = q_row - r * p.group;
    const int64_t head = (int64_t)(b * a.row_blocks + rb - a.e0) * p.n_kv_heads + kvh;
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.next = 0;
    if (SPLIT == 1 && !live) return;
    float m = -INFINITY, sum = 0.f, acc[V] = {};
    if (live) {
        const int64_t unit = head / a.heads;
        const int hs = (int)(head - unit * a.heads);
        const int4 at = __ldcg(p.ws_rows + (int64_t)b * p.q_rows + r);
        const int2 own = __ldcg(a.parts + unit);
        const int n1 = at.z, n = n1 + own.y - own.x + 1;
        const int64_t row1 = (int64_t)at.x + gh + (int64_t)kvh * n1 * at.y;  // + part * at.y
        // parts of the own keys: (unit + c) heads + hs, row `row`
        const int64_t row2 = ((unit + own.x) * a.heads + hs) * a.rb + row;
        const int64_t step2 = (int64_t)a.heads * a.rb;
        for (int x0 = warp % SPLIT; x0 < n; x0 += 32 * SPLIT) {
            const int x = x0 + lane * SPLIT;
            float2 lse = make_float2(-INFINITY, -INFINITY);
            if (x < n1) {
                lse = __ldcg(p.ws_lse + row1 + (int64_t)x * at.y);
            } else if (x < n) {
                lse.x = lse.y = __ldcg(a.lse + row2 + (x - n1) * step2) - a.held;
            }
            float mx = lse.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float m_new = fmaxf(m, mx), m_use = m_new == -INFINITY ? 0.f : m_new;
            const float old = m == -INFINITY ? 0.f : fast_exp2(m - m_use);
            const float fo = kPartWeight * fast_exp2(lse.x - m_use);
            float fs = kPartWeight * fast_exp2(lse.y - m_use);
            m = m_new;
#pragma unroll
            for (int d = 0; d < V; ++d) acc[d] *= fmaxf(old, kSmallest);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) fs += __shfl_xor_sync(0xffffffffu, fs, o);
            sum = sum * old + fs;
            const int in_round = min(32, (n - x0 + SPLIT - 1) / SPLIT);
            const int shared = max(0, min(in_round, (n1 - x0 + SPLIT - 1) / SPLIT));
            // the outputs of kBatch parts are asked for before one is used
            constexpr int kBatch = SPLIT == 1 ? 4 : 8;
            const uint16_t *src1 = p.ws_o + (row1 + (int64_t)x0 * at.y) * HD + lane * V;
            for (int k0 = 0; k0 < shared; k0 += kBatch) {
                uint2 raw[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const uint16_t *src = src1 + (int64_t)(k0 + i) * SPLIT * at.y * HD;
                    raw[i] = make_uint2(0u, 0u);
                    if (k0 + i < shared) {
                        if constexpr (V == 4)
                            raw[i] = __ldcg(reinterpret_cast<const uint2 *>(src));
                        else
                            raw[i].x = __ldcg(reinterpret_cast<const unsigned int *>(src));
                    }
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const float w = __shfl_sync(0xffffffffu, fo, (k0 + i) & 31);
                    if (k0 + i < shared)
#pragma unroll
                        for (int d = 0; d < V / 2; ++d) {
                            const float2 y = __half22float2(
                                *reinterpret_cast<const __half2 *>(d == 0 ? &raw[i].x : &raw[i].y));
                            acc[2 * d] += w * y.x;
                            acc[2 * d + 1] += w * y.y;
                        }
                }
            }
            for (int k0 = shared; k0 < in_round; k0 += kBatch / 2) {
                float4 raw[kBatch / 2];
#pragma unroll
                for (int i = 0; i < kBatch / 2; ++i) {
                    const float *src =
                        a.o + (row2 + (int64_t)(x0 + (k0 + i) * SPLIT - n1) * step2) * HD + lane * V;
                    if (k0 + i < in_round) {
                        if constexpr (V == 4) {
                            raw[i] = __ldcg(reinterpret_cast<const float4 *>(src));
                        } else {
                            const float2 y = __ldcg(reinterpret_cast<const float2 *>(src));
                            raw[i].x = y.x, raw[i].y = y.y;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < kBatch / 2; ++i) {
                    // no weight is 0: 0 times an infinite output would be NaN
                    const float w = fmaxf(__shfl_sync(0xffffffffu, fo, (k0 + i) & 31), kSmallest);
                    if (k0 + i < in_round) {
                        acc[0] += w * raw[i].x, acc[1] += w * raw[i].y;
                        if constexpr (V == 4) acc[2] += w * raw[i].z, acc[3] += w * raw[i].w;
                    }
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
    uint32_t *dst = reinterpret_cast<uint32_t *>(
        p.out + (((int64_t)b * p.q_rows + r) * p.n_q_heads + kvh * p.group + gh) * HD + lane * V);
#pragma unroll
    for (int d = 0; d < V / 2; ++d) dst[d] = pack_bf16x2(acc[2 * d] * inv, acc[2 * d + 1] * inv);
}

template <int FMT, int HD>
int launch_prefix(const Params &p, const CUtensorMap &tq, const CUtensorMap &tk,
                  const CUtensorMap &tv, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};  // a bit per device
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(configured.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e =
            cudaFuncSetAttribute(prefix_kernel<FMT, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)Cfg<FMT, HD>::kSmem);
        if (e != cudaSuccess) {
            note_cuda_error(e);
            return ATTN_ERR_CUDA;
        }
        configured.fetch_or(bit, std::memory_order_relaxed);
    }
    const unsigned grid = (unsigned)*std::max_element(p.sms, p.sms + kGroupSteps);
    const cudaError_t e = launch_pdl(prefix_kernel<FMT, HD>, dim3(grid), dim3(Cfg<FMT, HD>::kThreads),
                                     Cfg<FMT, HD>::kSmem, stream, tq, tk, tv, p);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int HD>
cudaError_t launch_merge(const MergeParams &p, bool split, cudaStream_t stream) {
    const int64_t rows = (int64_t)p.n_rows * p.n_kv_heads;
    return split ? launch_pdl(shared_merge_kernel<HD, 4>, dim3((unsigned)((rows + 1) / 2)), dim3(256),
                              0, stream, p)
                 : launch_pdl(shared_merge_kernel<HD, 1>, dim3((unsigned)((rows + 7) / 8)), dim3(256),
                              0, stream, p);
}

}  // namespace shr

int plan_shared(const attn_kv_cache *cache, int batch, int q_rows, int n_q_heads, int n_kv_heads,
                int head_dim, int max_seq_len, int window, SharedPlan *plan) {
    if (batch > shr::kMaxBatch) return ATTN_ERR_UNSUPPORTED;
    if (int rc = plan_attend(cache, batch, q_rows, n_q_heads, n_kv_heads, head_dim, max_seq_len,
                             window, 0, &plan->own, true);
        rc != ATTN_OK)
        return rc;
    // Parts of the shared keys: each row's first part or two, and those that units of at most
    // 256 rows are cut into beyond (at most one for every SM)
    const int64_t rows = (int64_t)batch * q_rows * n_q_heads;
    const int64_t parts = 2 * rows + (int64_t)2 * shr::kBM * device_sm_count();
    if (parts >= (int64_t(1) << 30)) return ATTN_ERR_SHAPE;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    plan->rows_offset = up(plan->own.workspace);
    plan->lse_offset = up(plan->rows_offset + (size_t)batch * q_rows * sizeof(int4));
    plan->o_offset = up(plan->lse_offset + (size_t)parts * sizeof(float2));
    plan->workspace = plan->o_offset + (size_t)parts * head_dim * 2;
    return ATTN_OK;
}

// The SMs that the shared part takes where `groups` groups share a prefix.  attend.cu's CTAs start at
// once on the others and follow on each that is left, so that the two parts run side by side.  Of the
// pieces that a unit (KV head, pair of tiles) can be cut into, as many as end soonest by the host's
// bounds (lengths are known on the device only): a piece takes 9 us and 1.65 a pair of tiles and 128
// keys (1.2 a single tile; over codes 2.4 and 1.6; 64 dims do best by the same: with three quarters
// of it for them 64 bf16 requests over 4,096 keys 34.4 us, so 31.8, and 16 over 14,449 24.1 and 25.8),
// an SM reads 36 bytes (28) of own keys a nanosecond.  On every SM first, the own keys after: 64 requests
// over 4,096 and 64 to 1,024 keys 67.8 us, side by side 47.8; 16 over 14,449 and up to 2,000 43.2 and
// 32.2; four E4M3 groups 68.9 and 61.3; two short requests the same.  Every group has a unit for each
// KV head: with what is right for one group, 64 requests in 32 groups of up to 128 shared keys took
// 285 us on 8 SMs, one piece after another (43 with their own number; 16 groups 148 and 37).  CTAs
// past one group's number look for themselves, which costs a batch of one group up to 1 us.
static int prefix_sms(int batch, int q_rows, int group, int n_kv_heads, int head_dim, int esize,
                      int max_seq_len, int max_prefix_len, int own_units, int groups) {
    const int sms = device_sm_count(), rt = shr::kBM / group;
    const int64_t pos = ((int64_t)batch * q_rows + groups - 1) / groups;  // of one of them
    const int64_t units =
        (((int64_t)batch * q_rows + 2 * rt - 1) / (2 * rt) + groups - 1) * n_kv_heads;
    if (units > sms / 2) return sms;
    const int64_t tiles = (max_prefix_len + 127) / 128;
    const double tile = esize == 2 ? (pos <= rt ? 1.2 : 1.65) : (pos <= rt ? 1.6 : 2.4);
    // microseconds of an SM: its rate, and a round trip or three for every change of unit
    const double own = 0.5 * batch * (double)(max_seq_len - max_prefix_len) * n_kv_heads *
                           head_dim * 2 * esize / (esize == 2 ? 36e3 : 28e3) +
                       (double)own_units * (esize == 2 ? 2.5 : 3.0);
    auto end_of = [&](uint32_t most_tiles, int k) {
        const double t = 9 + most_tiles * tile;
        // the own keys: on the other SMs until then, on all after
        const double left = own - t * (double)(sms - k * units);
        return t + (left > 0 ? 4 + left / sms : 0);
    };
    // ... of those about as good the most: late own keys cost less than a late shared part, which
    // is what a batch of several groups would have
    constexpr int kMost = 256;
    double ends[kMost + 1];
    const int ks = (int)std::min<int64_t>({sms / units, std::max<int64_t>(1, tiles), kMost});
    double least = 1e30;
    uint32_t before = 0;
    for (int k = 1; k <= ks; ++k) {
        const uint32_t most_tiles = ((uint32_t)tiles + k - 1) / k;
        ends[k] = most_tiles == before ? 1e30 : end_of(most_tiles, k);
        before = most_tiles;
        least = std::min(least, ends[k]);
    }
    int best = ks;
    while (best > 1 && ends[best] > 1.03 * least) --best;
    return (int)(best * units);
}

int launch_shared(const SharedPlan &plan, const void *q, const attn_kv_cache *cache, int n_rows,
                  const int32_t *seq_lens, const int32_t *positions, const int32_t *prefix_rows,
                  const int32_t *prefix_lens, int batch, int q_rows, int max_seq_len,
                  int max_prefix_len, int window, int n_q_heads, int n_kv_heads, int head_dim,
                  float scale, void *out, void *workspace, int32_t *err, cudaStream_t stream) {
    shr::Params p = {};
    const bool scaled = kv_scaled(cache->dtype), codes = cache->dtype != ATTN_KV_BF16;
    const int esize = codes ? 1 : 2;
    p.batch = batch;
    p.q_rows = q_rows;
    p.window = window;
    p.n_kv_heads = n_kv_heads;
    p.group = n_q_heads / n_kv_heads;
    p.rt = shr::kBM / p.group;
    // (the groups are known on the device only)
    for (int i = 0; i < shr::kGroupSteps && (1 << i) <= batch; ++i)
        p.sms[i] = prefix_sms(batch, q_rows, p.group, n_kv_heads, head_dim, esize, max_seq_len,
                              std::min(max_prefix_len, max_seq_len),
                              plan.own.entries * (n_kv_heads / plan.own.heads), 1 << i);
    p.n_rows = n_rows;
    p.slots_per_seq = cache->slots_per_seq;
    p.block_size = cache->block_size;
    p.max_blocks = cache->max_blocks_per_seq;
    p.paged = cache->kind == ATTN_CACHE_PAGED;
    p.num_pages = p.paged ? (int)(cache->num_slots / cache->block_size) : 0;
    p.cap = p.paged ? max_seq_len : std::min(max_seq_len, cache->slots_per_seq);
    p.prefix_cap = std::min(max_prefix_len, p.cap);
    p.head_major = cache->layout == ATTN_LAYOUT_BHSD;
    p.block_table = p.paged ? cache->block_table : nullptr;
    p.seq_lens = seq_lens;
    p.positions = positions;
    p.prefix_rows = prefix_rows;
    p.prefix_lens = prefix_lens;
    p.k = static_cast<const uint8_t *>(cache->k);
    p.v = static_cast<const uint8_t *>(cache->v);
    p.ks = scaled ? cache->k_scale : nullptr;
    p.vs = scaled ? cache->v_scale : nullptr;
    if (scaled)
        while ((1 << p.scale_shift) < cache->scale_block) ++p.scale_shift;
    p.place = kv_place(cache, n_kv_heads, head_dim, esize);
    p.scale_log2 = scale * 1.4426950408889634f;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.ws_rows = reinterpret_cast<int4 *>(ws + plan.rows_offset);
    p.ws_lse = reinterpret_cast<float2 *>(ws + plan.lse_offset);
    p.ws_o = reinterpret_cast<uint16_t *>(ws + plan.o_offset);
    p.err = err;
    // the largest power of two of keys that lie together wherever a tile begins; TMA boxes of
    // less than 8 would not begin on a swizzle's period
    p.box_rows = shr::kBN;
    if (p.paged) {
        p.box_rows = std::min(cache->block_size & -cache->block_size, shr::kBN);
        if (p.box_rows < 8) p.box_rows = 0;
        int l = 0;
        while ((int64_t(1) << l) < cache->block_size) ++l;
        p.page_shift = 31 + l;
        p.page_mul = (uint32_t)((uint64_t(1) << p.page_shift) / cache->block_size + 1);
    }

    CUtensorMap tq, tk = {}, tv = {};
    const uint64_t dq[3] = {(uint64_t)head_dim, (uint64_t)n_q_heads, (uint64_t)batch * q_rows};
    const uint64_t sq[2] = {(uint64_t)head_dim * 2, (uint64_t)n_q_heads * head_dim * 2};
    const uint32_t bq[3] = {64, (uint32_t)p.group, (uint32_t)p.rt};
    bool ok = encode_tensor_map(&tq, q, 3, dq, sq, bq, true);
    if (p.box_rows > 0) {
        const uint64_t row = (uint64_t)head_dim * esize;
        uint64_t d[3], s[2];
        if (p.head_major) {
            const uint64_t rows = p.paged ? cache->block_size : cache->slots_per_seq;
            d[0] = head_dim, d[1] = rows, d[2] = (uint64_t)cache->num_slots / rows * n_kv_heads;
            s[0] = row, s[1] = rows * row;
        } else {
            d[0] = (uint64_t)n_kv_heads * head_dim, d[1] = cache->num_slots, d[2] = 1;
            s[0] = n_kv_heads * row, s[1] = (uint64_t)cache->num_slots * n_kv_heads * row;
        }
        p.map_rows = (int)d[1];
        const uint32_t box[3] = {codes ? (uint32_t)head_dim : 64u, (uint32_t)p.box_rows, 1};
        const bool swizzle = !codes || head_dim == 128;
        ok = ok && encode_tensor_map(&tk, cache->k, 3, d, s, box, swizzle, codes) &&
             encode_tensor_map(&tv, cache->v, 3, d, s, box, swizzle, codes);
    }
    if (!ok) {
        note_cuda_error(cudaErrorInvalidValue);
        return ATTN_ERR_CUDA;
    }
    int rc;
    if (cache->dtype == ATTN_KV_BF16)
        rc = head_dim == 128 ? shr::launch_prefix<shr::kBF16, 128>(p, tq, tk, tv, stream)
                             : shr::launch_prefix<shr::kBF16, 64>(p, tq, tk, tv, stream);
    else if (cache->dtype == ATTN_KV_INT8_SCALED)
        rc = head_dim == 128 ? shr::launch_prefix<shr::kINT8, 128>(p, tq, tk, tv, stream)
                             : shr::launch_prefix<shr::kINT8, 64>(p, tq, tk, tv, stream);
    else
        rc = head_dim == 128 ? shr::launch_prefix<shr::kE4M3, 128>(p, tq, tk, tv, stream)
                             : shr::launch_prefix<shr::kE4M3, 64>(p, tq, tk, tv, stream);
    if (rc != ATTN_OK) return rc;

    shr::MergeParams m = {};
    m.ws_rows = p.ws_rows;
    m.ws_lse = p.ws_lse;
    m.ws_o = p.ws_o;
    m.out = static_cast<__nv_bfloat16 *>(out);
    m.q_rows = q_rows;
    m.rows = q_rows * p.group;
    m.n_q_heads = n_q_heads;
    m.n_kv_heads = n_kv_heads;
    m.group = p.group;
    // Four warps a row where rows lie in many parts (if all requests are one group) and are few:
    // 16 requests of 28/4 heads over 14,449 keys 32.2 us, with one warp 42.4; 64 of 32/8 over 4,096
    // 47.8 with one, 55.8 with four; 256 over 32,768 155 and 188
    const int64_t pairs = ((int64_t)batch * q_rows + 2 * p.rt - 1) / (2 * p.rt);
    const bool split = p.sms[0] > 8 * n_kv_heads * pairs &&
                       (int64_t)batch * q_rows * n_q_heads <= (int64_t)p.sms[0] * 16;
    for (int e0 = 0; e0 < plan.own.entries; e0 += plan.own.per_launch) {
        rc = launch_attend_parts(plan.own, e0, prefix_lens, p.prefix_cap, q, cache, seq_lens,
                                 positions, q_rows, max_seq_len, window, n_q_heads, n_kv_heads,
                                 head_dim, scale, out, workspace, err, stream, e0 == 0, &m.own);
        if (rc != ATTN_OK) return rc;
        // rows of entries e0 .. e0 + n_entries - 1 (a request's last block may be short)
        auto row_of = [&](int e) {
            const int b = e / plan.own.row_blocks;
            return b * m.rows + (e - b * plan.own.row_blocks) * m.own.rb;
        };
        m.first_row = row_of(e0);
        m.n_rows = row_of(e0 + m.own.n_entries) - m.first_row;
        const cudaError_t e = head_dim == 128 ? shr::launch_merge<128>(m, split, stream)
                                              : shr::launch_merge<64>(m, split, stream);
        if (e != cudaSuccess) return ATTN_ERR_CUDA;
    }
    return ATTN_OK;
}

}  // namespace gqa
