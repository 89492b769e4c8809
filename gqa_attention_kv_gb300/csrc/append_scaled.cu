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
// A copy with arithmetic: HBM is its floor.  The rows of a call that lie in one block
// are a run; nothing is shared between the warps that write different runs, so there
// is no order to depend on.  Two kernels, by the length of runs to expect:
//   * runs by warps: a warp takes whole runs, reading its rows once where they fit its
//     registers (16 rows of 128, 32 of 64).  Steps, and prompts in blocks of 16:
//     14,449 rows of 4 x 128 in 10.9 us (4.1 TB/s; issue-bound: unpacking, scaling and
//     packing 16-bit values), 64 single rows of 8 x 128 in 2.9 us.
//     Of many rows a warp has 16, and the short runs among them are taken all at a time,
//     a lane a row: single rows of 1,024 requests 5.8 us (19.1 one after another, 12.9 by
//     a warp each), of 4,096 10.9 (40.6).
//   * runs by CTAs: 64 rows (128 for blocks of 128) of one tensor and head, 16 a warp,
//     in registers; the rows' maxima meet in shared memory, each warp finds the ends of
//     the runs that its rows belong to in the slots around them and encodes its own
//     rows.  Rows of a run outside the CTA are read again for their maximum.  The warp
//     with the run's first row stores the scale and, where it grew, recodes the
//     block's slots that the run does not write; a warp elsewhere that reads the scale
//     after it was stored comes to the same new scale.  Many rows in longer blocks:
//     14,449 rows of 4 x 128 in blocks of 32 17.7 us (27 by warps), of 64 18.3 (39), of
//     128 19.3 (61); in blocks of 16 it would take 17.4.
// Rows of a block in another order than their slots', or with skipped rows among
// them, are an irregular run: written alone by the warp that has its first row.
// Skipped rows beside a run (a padded batch) are looked through 64 at a time for the
// row that says whether the run goes on: 14,449 rows padded to 16,384, into one cache again
// and again, take 17 us in blocks of 16 and 23 to 25 in longer ones (9.6 and 14.3 to 16.1
// without padding), one row of 4,001 19 to 22; one skipped row after another, each walked
// again by the warp of the run, 315, 377 to 414 and 635 to 720 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "kernels.h"
#include "ptx.cuh"

namespace gqa {
namespace {

constexpr float kScaleFloor = 5.421010862427522e-20f;  // 2^-64
constexpr int kPasses = 8;   // row groups that a warp of the runs kernel holds in registers
constexpr int kMaxWindow = 16, kMaxBlock = 128;
constexpr int64_t kNone = INT64_MIN, kBad = -1;        // rows outside the call; slots outside the cache

struct ScaledParams {
    const uint4 *k_new, *v_new;
    const float *k_ref;
    const int64_t *slots;
    int64_t n;
    uint8_t *k, *v;
    float *ks, *vs;
    int64_t num_slots;
    int shift;  // log2 of the slots of a block
    int window;  // rows of a warp (runs kernel)
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

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Codes of four values.  CLAMP false: |x r| <= 127 (1 + 2^-22), as finite rows have
// under a scale of their own maximum.
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

// The codes of a block's slots, times `by`, but for slots lo .. hi - 1.
template <bool INT8, int HD>
__device__ __forceinline__ void recode(const ScaledParams &p, uint8_t *cache, int h, int64_t block,
                                       float by, int64_t lo, int64_t hi) {
    constexpr int kL = HD / 16, kR = 32 / kL;  // 16 codes a lane
    const int lane = threadIdx.x & 31;
    for (int s0 = 0; s0 < (1 << p.shift); s0 += kR) {
        const int64_t s = (block << p.shift) + s0 + lane / kL;
        if (s0 + lane / kL >= (1 << p.shift) || (s >= lo && s < hi)) continue;
        uint4 *c = reinterpret_cast<uint4 *>(cache + p.place.head_offset(s, h) +
                                             (lane & (kL - 1)) * 16);
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
    __syncwarp();
}

// From row i on (DIR 1; -1: back from it), past the rows without a slot of the cache, 64
// of them a step: the slot of the first that has one, kNone where the call ends before.
template <int DIR>
__device__ __forceinline__ int64_t next_slot(const ScaledParams &p, int64_t &i) {
    constexpr int kLoads = 2;
    const int lane = threadIdx.x & 31;
    for (; i >= 0 && i < p.n; i += DIR * 32 * kLoads) {
        int64_t s[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int64_t row = i + DIR * (32 * u + lane);
            s[u] = row >= 0 && row < p.n ? __ldg(p.slots + row) : kBad;
        }
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const uint32_t found = __ballot_sync(0xffffffffu, s[u] >= 0 && s[u] < p.num_slots);
            if (found != 0) {
                i += DIR * (32 * u + __ffs(found) - 1);
                return __shfl_sync(0xffffffffu, s[u], __ffs(found) - 1);
            }
        }
    }
    return kNone;
}

// s' from the scale held (0 where the block starts anew) and the rows' maximum.
template <bool INT8>
__device__ __forceinline__ float new_scale(float held, float amax) {
    return fmaxf(fmaxf(held, __fdiv_rn(amax, INT8 ? 127.f : 448.f)), kScaleFloor);
}

// The eight values of a lane's piece of a row, less ref's.
__device__ __forceinline__ void piece_values(const uint4 &w, const float *ref, float *f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = __uint_as_float(u[e] << 16);
        f[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
    }
    if (ref != nullptr)
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __fsub_rn(f[e], __ldg(ref + e));
}

// The largest magnitude of a row, NaN if it holds one, in all of the row's lanes.
template <int LANES>
__device__ __forceinline__ float row_max(const uint4 &w, const float *ref) {
    float m;
    if (ref == nullptr) {
        uint32_t a = max_nan_bf16x2(max_nan_bf16x2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                    max_nan_bf16x2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1)
            a = max_nan_bf16x2(a, __shfl_xor_sync(0xffffffffu, a, o));
        m = max_nan(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
    } else {
        float f[8];
        piece_values(w, ref, f);
        m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(f[e]));
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    return m;
}

// Short runs of a warp's 16 rows, all at a time, a lane a row (lane 16 the row behind
// them): those that begin at one of `starts`, end among the rows and hold finite values
// in slots of the cache.  x: the rows; slot < 0: no row (kNone) or a skipped one; amax:
// the row's largest magnitude; held: its block's scale.  Returns the rows written.
template <bool INT8, int HD>
__device__ __forceinline__ uint32_t append_short_runs(const ScaledParams &p, uint8_t *cache,
                                                      float *scales, const float *ref, int h,
                                                      const uint4 *x, int64_t slot, float amax,
                                                      float held, uint32_t starts) {
    constexpr int kLanes = HD / 8, kRows = 32 / kLanes;
    const int lane = threadIdx.x & 31, heads = p.place.n_kv_heads;
    const int64_t block = slot >> p.shift, next = __shfl_down_sync(0xffffffffu, slot, 1);
    const bool good = slot >= 0;
    // rows whose next row belongs to the same run, or is skipped
    const uint32_t same =
        __ballot_sync(0xffffffffu, good && lane < 16 && next >= 0 && (next >> p.shift) == block);
    const uint32_t skipped = __ballot_sync(0xffffffffu, slot < 0 && slot != kNone);
    const int last = lane + __ffs(~(same >> lane)) - 1;                   // of this lane's run
    const uint32_t firsts = ~(same << 1) & (0xffffffffu >> (31 - lane));  // up to this lane
    const int first = 31 - __clz(firsts);
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
        const float t = __shfl_down_sync(0xffffffffu, amax, o);
        if (lane + o <= last) amax = max_nan(amax, t);
    }
    amax = __shfl_sync(0xffffffffu, amax, first);
    const bool mine = good && lane < 16 && last < 16 && !((skipped >> (last + 1)) & 1u) &&
                      ((starts >> first) & 1u) && amax < INFINITY;
    const uint32_t zero = __ballot_sync(0xffffffffu, good && (slot & ((1 << p.shift) - 1)) == 0);
    const bool fresh = ((zero >> first) & ((2u << (last - first)) - 1u)) != 0;
    held = fresh ? 0.f : fmaxf(held, 0.f);
    const float now = new_scale<INT8>(held, amax), r = __frcp_rn(now), by = __fmul_rn(held, r);
    const uint32_t rows = __ballot_sync(0xffffffffu, mine);
    uint32_t grown = __ballot_sync(0xffffffffu, mine && lane == first && held > 0.f && now > held);
    while (grown != 0) {
        const int a = __ffs(grown) - 1;
        grown &= grown - 1;
        recode<INT8, HD>(p, cache, h, __shfl_sync(0xffffffffu, block, a),
                         __shfl_sync(0xffffffffu, by, a), 0, 0);
    }
    __syncwarp();
    if (mine && lane == first) scales[block * heads + h] = now;
#pragma unroll
    for (int u = 0; u < 16 / kRows; ++u) {
        const int row = u * kRows + lane / kLanes;
        const float rr = __shfl_sync(0xffffffffu, r, row);
        const int64_t to = __shfl_sync(0xffffffffu, slot, row);
        if (!((rows >> row) & 1u)) continue;
        float f[8];
        piece_values(x[u], ref, f);
        *reinterpret_cast<uint2 *>(cache + p.place.head_offset(to, h) +
                                   (lane & (kLanes - 1)) * 8) =
            make_uint2(encode4<INT8, false>(f, rr), encode4<INT8, false>(f + 4, rr));
    }
    __syncwarp();
    return rows;
}

// Runs by warps: a warp takes the runs that start among its rows (one to sixteen),
// whatever their length, alone.  A run that ends among these rows stays in registers
// between its maximum and its codes.
// SHORT: short runs are taken together where a warp's rows hold more than one.
template <bool INT8, int HD, bool SHORT>
__global__ void __launch_bounds__(128, 6) kv_append_runs_kernel(const ScaledParams p) {
    constexpr int kLanes = HD / 8;           // lanes of a row: 16 bytes of bf16, 8 codes each
    constexpr int kRows = 32 / kLanes;       // rows of a pass
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
    const bool mine = lane >= 1 && lane <= p.window && seen < p.n;
    bool far = false;  // the row before is skipped: rows that are do not end a run
    if (mine) {
        if (good(my_slot)) {
            far = seen > 0 && !good(before);
            start = !far && (seen == 0 || (before >> p.shift) != (my_slot >> p.shift));
        } else if (rem == 0) {
            report_error(p.err, ATTN_ERR_BOUNDS);
        }
    }
    for (uint32_t rows = __ballot_sync(0xffffffffu, far); rows != 0; rows &= rows - 1) {
        const int l = __ffs(rows) - 1;
        int64_t j = first_row - 1 + l - 2;
        const int64_t t = next_slot<-1>(p, j);
        if (lane == l) start = t == kNone || (t >> p.shift) != (my_slot >> p.shift);
    }
    // the scales that the runs' blocks hold, all in one trip
    const float my_scale = start ? scales[(my_slot >> p.shift) * heads + h] : 0.f;
    uint32_t starts = __ballot_sync(0xffffffffu, start);
    bool intact = true;  // x holds the window's rows
    if (SHORT && (starts & (starts - 1)) != 0) {
        float amax = 0.f;
#pragma unroll
        for (int u = 0; u < kMaxWindow / kRows; ++u) {
            const float m = __shfl_sync(0xffffffffu, row_max<kLanes>(x[u], ref),
                                        lane % kRows * kLanes);
            if (lane / kRows == u) amax = m;
        }
        const int64_t s = __shfl_down_sync(0xffffffffu, my_slot, 1);
        const float held = __shfl_down_sync(0xffffffffu, my_scale, 1);
        const int64_t row = first_row + lane;
        const int64_t slot = row >= p.n ? kNone : good(s) ? s : kBad;
        // (a run's first lane has its scale)
        const uint32_t first = (starts >> 1) & (0xffffffffu >> (31 - lane));
        const float of_run = __shfl_sync(0xffffffffu, held, first == 0 ? 0 : 31 - __clz(first));
        starts &= ~(append_short_runs<INT8, HD>(p, cache, scales, ref, h, x, slot, amax, of_run,
                                                starts >> 1) << 1);
    }
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
            const uint32_t rows = __ballot_sync(
                0xffffffffu, lane >= at_lane && lane < stop && good(my_slot));
            int64_t end = first_row - 1 + 32 - __clz(rows);  // behind its last row
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
                const uint32_t some = __ballot_sync(0xffffffffu, lane < take && good(s));
                if (some != 0) end = i1 + 32 - __clz(some);
                i1 += take;
                if (take < 32) break;
                if (some == 0 && next_slot<1>(p, i1) >> p.shift != block) break;
            }
            i1 = end;
        }
        auto slot_of = [&](int64_t i) -> int64_t {  // all lanes together
            const int64_t l = i - (first_row - 1);
            const int64_t s = __shfl_sync(0xffffffffu, my_slot, (int)(l & 31));
            return l < 32 ? s : __ldg(p.slots + min(i, p.n - 1));
        };
        auto load = [&](int64_t base) { fetch(base, i1, true); };
        auto values = [&](const uint4 &w, float *f) { piece_values(w, ref, f); };
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
                                        (good(my_slot) && my_slot == slot0 + (lane - at_lane)));
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
        const float now = new_scale<INT8>(held, amax);
        const float r = __frcp_rn(now);
        // the block's earlier codes (the run's rows among them are written below)
        if (held > 0.f && now > held)
            recode<INT8, HD>(p, cache, h, block, __fmul_rn(held, r), 0, 0);
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

// Runs by CTAs: for long runs.  See the head of this file.
template <bool INT8, int HD, int W>
__global__ void __launch_bounds__(W * 32, 24 / W)
    kv_append_blocks_kernel(const __grid_constant__ ScaledParams p) {
    constexpr int kLanes = HD / 8;                // lanes of a row: 16 bytes of bf16, 8 codes each
    constexpr int kRows = 32 / kLanes;            // rows of a pass
    constexpr int kPasses = kMaxWindow / kRows;   // of a warp's 16 rows
    __shared__ int64_t sm_slot[2 * kMaxBlock + W * kMaxWindow];
    __shared__ float sm_max[W * kMaxWindow];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int heads = p.place.n_kv_heads, sb = 1 << p.shift;
    const int64_t group = blockIdx.x / (2 * heads);
    const int rem = (int)(blockIdx.x - group * (2 * heads)), tensor = rem / heads;
    const int h = rem - tensor * heads;
    const int cta_rows = W * kMaxWindow;
    const int64_t row0 = group * cta_rows;        // of the CTA
    const int w0 = warp * kMaxWindow;               // this warp's first row, in the CTA's
    const int n_cta = (int)min((int64_t)cta_rows, p.n - row0);
    const uint4 *src = tensor == 0 ? p.k_new : p.v_new;
    uint8_t *cache = tensor == 0 ? p.k : p.v;
    float *scales = tensor == 0 ? p.ks : p.vs;
    const int my_r = lane / kLanes, piece = lane & (kLanes - 1);
    const float *ref = tensor == 0 && p.k_ref != nullptr ? p.k_ref + h * HD + piece * 8 : nullptr;

    // ---- this warp's rows, and the slots of the CTA's rows and a block's length around
    uint4 x[kPasses];
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
        const int r = w0 + my_r + u * kRows;
        x[u] = make_uint4(0u, 0u, 0u, 0u);
        if (my_r + u * kRows < kMaxWindow && r < n_cta)
            x[u] = __ldg(src + ((row0 + r) * heads + h) * kLanes + piece);
    }
    for (int i = threadIdx.x; i < cta_rows + 2 * sb; i += W * 32) {
        const int64_t row = row0 - sb + i;
        int64_t s = row >= 0 && row < p.n ? __ldg(p.slots + row) : kNone;
        if (s != kNone && (s < 0 || s >= p.num_slots)) {
            s = kBad;
            if (rem == 0 && i >= sb && i < sb + cta_rows) report_error(p.err, ATTN_ERR_BOUNDS);
        }
        sm_slot[i] = s;
    }
    __syncthreads();
    auto slot = [&](int r) { return sm_slot[sb + r]; };  // of the CTA's row r, -sb <= r < rows + sb

    // ---- the rows' maxima, and the scales of their blocks
    const int64_t my_slot = lane < kMaxWindow && w0 + lane < n_cta ? slot(w0 + lane) : kNone;
    const float my_scale = my_slot >= 0 ? scales[(my_slot >> p.shift) * heads + h] : 0.f;
    auto values = [&](const uint4 &w, float *f) { piece_values(w, ref, f); };
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
        const float m = row_max<kLanes>(x[u], ref);
        if (piece == 0 && my_r + u * kRows < kMaxWindow) sm_max[w0 + my_r + u * kRows] = m;
    }
    __syncthreads();

    // ---- this warp's pieces: rows in consecutive slots of one block
    const int64_t before = lane >= 1 && lane < kMaxWindow ? slot(w0 + lane - 1) : kNone;
    uint32_t starts = __ballot_sync(0xffffffffu, my_slot >= 0 &&
                                                     (my_slot != before + 1 || before < 0 ||
                                                      (my_slot & (sb - 1)) == 0));
    const uint32_t good = __ballot_sync(0xffffffffu, my_slot >= 0), pieces = starts;
    if (__popc(starts) > 2) {
        // more than a block's end and another's beginning: the short runs together, a lane
        // a row
        const int64_t s = lane <= kMaxWindow ? slot(w0 + lane) : kNone;
        const int64_t b4 = lane < kMaxWindow ? slot(w0 + lane - 1) : kNone;
        const uint32_t apart = __ballot_sync(
            0xffffffffu, s >= 0 && (b4 == kNone || (b4 >= 0 && (b4 >> p.shift) != (s >> p.shift))));
        starts &= ~append_short_runs<INT8, HD>(
            p, cache, scales, ref, h, x, s, lane < kMaxWindow ? sm_max[w0 + lane] : 0.f, my_scale,
            apart);
    }
    while (starts != 0) {
        const int a = __ffs(starts) - 1;  // the piece: rows w0 + a .. w0 + b - 1
        starts &= starts - 1;
        const uint32_t ends = (pieces | ~good) & (0xfffffffeu << a);
        const int b = ends == 0 ? 32 : __ffs(ends) - 1;
        const int64_t s_a = slot(w0 + a), block = s_a >> p.shift;
        const int off = (int)(s_a & (sb - 1));
        // rows before and behind it in the consecutive slots of the block
        int r0 = w0 + a, r1 = w0 + b;
        for (int j0 = 0; j0 < off; j0 += 32) {
            const int j = j0 + lane + 1;
            const uint32_t no = __ballot_sync(0xffffffffu, j > off || slot(w0 + a - j) != s_a - j);
            const int run = no == 0 ? 32 : __ffs(no) - 1;
            r0 -= run;
            if (run < 32) break;
        }
        const int room = sb - off - (b - a);  // slots of the block behind the piece
        for (int j0 = 0; j0 < room; j0 += 32) {
            const int j = j0 + lane;
            const uint32_t no = __ballot_sync(
                0xffffffffu, j >= room || slot(w0 + b + j) != s_a + (b - a) + j);
            const int run = no == 0 ? 32 : __ffs(no) - 1;
            r1 += run;
            if (run < 32) break;
        }
        // regular: no other row of the block beside it, also not behind rows without a slot
        auto other_block = [&](int64_t s) { return s == kNone || (s >= 0 && (s >> p.shift) != block); };
        bool regular = other_block(slot(r0 - 1)) && other_block(slot(r1));
        if (!regular && (slot(r0 - 1) == kBad || slot(r1) == kBad)) {
            int64_t i = row0 + r0 - 1;
            regular = other_block(next_slot<-1>(p, i));
            i = row0 + r1;
            if (regular) regular = other_block(next_slot<1>(p, i));
        }
        if (regular) {
            const int64_t first = s_a - (w0 + a - r0);  // slot of the run's first row
            const bool fresh = (first & (sb - 1)) == 0;
            float amax = 0.f;
            for (int r = max(r0, 0) + lane; r < min(r1, n_cta); r += 32)
                amax = max_nan(amax, sm_max[r]);
            auto other = [&](int lo, int hi) {  // rows of the run that the CTA does not have
#pragma unroll 4
                for (int r = lo; r < hi; r += kRows) {
                    uint4 w = make_uint4(0u, 0u, 0u, 0u);
                    if (r + my_r < hi)
                        w = __ldg(src + ((row0 + r + my_r) * heads + h) * kLanes + piece);
                    else if (ref != nullptr)  // (its distance from the reference is no maximum)
                        w = __ldg(src + ((row0 + lo) * heads + h) * kLanes + piece);
                    amax = max_nan(amax, row_max<kLanes>(w, ref));
                }
            };
            other(r0, min(0, r1));
            other(max(n_cta, r0), r1);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const bool finite = amax < INFINITY;
            bool nan = false;
            if (!finite) {  // again, without the elements that are not
                amax = 0.f;
                for (int r = r0 + my_r; r < r1; r += kRows) {
                    float f[8];
                    values(__ldg(src + ((row0 + r) * heads + h) * kLanes + piece), f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float m = fabsf(f[e]);
                        nan |= m != m;
                        amax = fmaxf(amax, m < INFINITY ? m : 0.f);
                    }
                }
                __syncwarp();
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                if (INT8 && nan) report_error(p.err, ATTN_ERR_UNSUPPORTED);  // INT8 has no NaN: 0
            }
            const float held = fresh ? 0.f : fmaxf(__shfl_sync(0xffffffffu, my_scale, a), 0.f);
            const float now = new_scale<INT8>(held, amax), r = __frcp_rn(now);
            if (r0 == w0 + a) {  // the run's first row is this warp's
                if (held > 0.f && now > held)
                    recode<INT8, HD>(p, cache, h, block, __fmul_rn(held, r), first,
                                     first + (r1 - r0));
                if (lane == 0) scales[block * heads + h] = now;
            }
            const int64_t row_bytes = (int64_t)p.place.head_bytes * (p.place.rows == 0 ? heads : 1);
            uint8_t *dst = cache + p.place.head_offset(s_a, h) + (my_r - a) * row_bytes + piece * 8;
#pragma unroll
            for (int u = 0; u < kPasses; ++u, dst += kRows * row_bytes) {
                if (my_r + u * kRows < a || my_r + u * kRows >= b) continue;
                float f[8];
                values(x[u], f);
                uint2 c;
                if (finite) {
                    c = make_uint2(encode4<INT8, false>(f, r), encode4<INT8, false>(f + 4, r));
                } else {
                    if (INT8)
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = f[e] == f[e] ? f[e] : 0.f;
                    c = make_uint2(encode4<INT8, true>(f, r), encode4<INT8, true>(f + 4, r));
                }
                *reinterpret_cast<uint2 *>(dst) = c;
            }
            __syncwarp();
            continue;
        }
        // ---- an irregular run: written by the warp that has its first row
        const int64_t i0 = row0 + w0 + a;
        int64_t i = i0 - 1;
        int64_t s = next_slot<-1>(p, i);
        if (s != kNone && (s >> p.shift) == block) continue;  // its first row is another
        auto in_block = [&](int64_t t) { return t >= 0 && t < p.num_slots && (t >> p.shift) == block; };
        int64_t i1 = i0;  // behind its last row
        for (i = i0;;) {
            if (s = next_slot<1>(p, i); s == kNone || (s >> p.shift) != block) break;
            s = i + lane < p.n ? __ldg(p.slots + i + lane) : kBad;
            const uint32_t past = __ballot_sync(
                0xffffffffu, s >= 0 && s < p.num_slots && (s >> p.shift) != block);
            const uint32_t rows = __ballot_sync(0xffffffffu, in_block(s)) &
                                  (past == 0 ? 0xffffffffu : (past & -past) - 1u);
            i1 = i + 32 - __clz(rows);
            if (past != 0) break;
            i += 32;
        }
        float amax = 0.f;
        bool fresh = false, nan = false;
        for (int64_t r = i0 + my_r; r < i1; r += kRows) {
            s = __ldg(p.slots + r);
            if (!in_block(s)) continue;
            fresh |= (s & (sb - 1)) == 0;
            float f[8];
            values(__ldg(src + (r * heads + h) * kLanes + piece), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float m = fabsf(f[e]);
                nan |= m != m;
                amax = fmaxf(amax, m < INFINITY ? m : 0.f);
            }
        }
        __syncwarp();
        fresh = __any_sync(0xffffffffu, fresh);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float held = fresh ? 0.f : fmaxf(__shfl_sync(0xffffffffu, my_scale, a), 0.f);
        const float now = new_scale<INT8>(held, amax), r = __frcp_rn(now);
        // all of the block's slots: the run's are written afterwards
        if (held > 0.f && now > held)
            recode<INT8, HD>(p, cache, h, block, __fmul_rn(held, r), 0, 0);
        if (INT8 && nan) report_error(p.err, ATTN_ERR_UNSUPPORTED);
        __syncwarp();
        if (lane == 0) scales[block * heads + h] = now;
        for (int64_t t = i0 + my_r; t < i1; t += kRows) {
            s = __ldg(p.slots + t);
            if (!in_block(s)) continue;
            float f[8];
            values(__ldg(src + (t * heads + h) * kLanes + piece), f);
            if (INT8)
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = f[e] == f[e] ? f[e] : 0.f;
            *reinterpret_cast<uint2 *>(cache + p.place.head_offset(s, h) + piece * 8) =
                make_uint2(encode4<INT8, true>(f, r), encode4<INT8, true>(f + 4, r));
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
    const int64_t per_row = 2ll * n_kv_heads;
    const bool int8 = cache->dtype == ATTN_KV_INT8_SCALED;
    auto run = [&](auto kernel, int64_t blocks, int threads) {
        if (blocks >= (int64_t(1) << 31)) return (int)ATTN_ERR_SHAPE;
        return launch_pdl(kernel, dim3((unsigned)blocks), dim3(threads), 0, stream, p) == cudaSuccess
                   ? (int)ATTN_OK
                   : (int)ATTN_ERR_CUDA;
    };
    // While the GPU holds a warp for every row and head at once, each has one.  Past that
    // warps have 16 rows (of blocks longer than 16: CTAs, a prompt's runs being long).
    // 8 x 128: 512 single rows 8.8 us by a warp each, 5.7 by warps of 16; a prompt of 512
    // 9.4 and 3.6; 1,024 single rows 5.8, a prompt 3.7 to 4.2.
    const bool many = n * per_row > (int64_t)device_sm_count() * 24;
    if (many && cache->scale_block > 16) {
        const int w = cache->scale_block > 64 ? 8 : 4;
        const int64_t blocks = (n + w * kMaxWindow - 1) / (w * kMaxWindow) * per_row;
        if (head_dim == 128)
            return w == 4 ? run(int8 ? kv_append_blocks_kernel<true, 128, 4>
                                     : kv_append_blocks_kernel<false, 128, 4>, blocks, 128)
                          : run(int8 ? kv_append_blocks_kernel<true, 128, 8>
                                     : kv_append_blocks_kernel<false, 128, 8>, blocks, 256);
        return w == 4 ? run(int8 ? kv_append_blocks_kernel<true, 64, 4>
                                 : kv_append_blocks_kernel<false, 64, 4>, blocks, 128)
                      : run(int8 ? kv_append_blocks_kernel<true, 64, 8>
                                 : kv_append_blocks_kernel<false, 64, 8>, blocks, 256);
    }
    p.window = many ? kMaxWindow : 1;
    const int64_t warps = (n + p.window - 1) / p.window * per_row, blocks = (warps + 3) / 4;
    // Past a round and a half of such warps the rows are taken for a prompt's.  At every
    // size a prompt is a little faster without short runs, by the registers they take, and
    // single rows several times slower: 9,000 rows of 4 x 128 as a prompt 6.9 us without
    // and 7.4 with them, single 42 and 11; 14,449 rows 10.9 and 12.1, 60 and 16.
    if (many && 2 * warps <= (int64_t)device_sm_count() * 24 * 3)
        return head_dim == 128 ? run(int8 ? kv_append_runs_kernel<true, 128, true>
                                          : kv_append_runs_kernel<false, 128, true>, blocks, 128)
                               : run(int8 ? kv_append_runs_kernel<true, 64, true>
                                          : kv_append_runs_kernel<false, 64, true>, blocks, 128);
    return head_dim == 128 ? run(int8 ? kv_append_runs_kernel<true, 128, false>
                                      : kv_append_runs_kernel<false, 128, false>, blocks, 128)
                           : run(int8 ? kv_append_runs_kernel<true, 64, false>
                                      : kv_append_runs_kernel<false, 64, false>, blocks, 128);
}

}  // namespace gqa
