// Device helpers shared by the kernels of the paged KV cache.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "paged.h"

namespace tam {

// e4m3 rows carry one power-of-two scale per token and KV head, kept as its biased
// exponent (E8M0): scale = 2^(byte - 127), 255 = NaN.
constexpr int kScaleBias = 127;
constexpr int kScaleExpMin = -100, kScaleExpMax = 120;
constexpr uint32_t kScaleNan = 255;
// The smallest scale that a write gives, and so the scale of a row of zeros.
constexpr uint32_t kScaleLeast = kScaleBias + kScaleExpMin;
// The 16-bit products keep O in units of a power of two that follows the scales of V, and P in
// fp16 next to it: a probability below 2^-21 of the row's largest is off by up to 2^-32 of it, times
// the largest V around.  An item's scales may span 2^kSpan for that: beside the V row of the
// largest probability (224 2^low or more) such a key (448 2^high or less) is off by less than
// 2^(kSpan - 31) = 2^-15, to bf16's 2^-9.  (The changes of the unit are exact then, too: P V sums
// over 2^30 keys to less than 2^61, and its smallest product is 2^-48.)
constexpr int kSpan = 16;

// 2^(byte - 127) in fp32, NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return __uint_as_float(byte == kScaleNan ? 0x7fc00000u : byte ? byte << 23 : 0x00400000u);
}

// 2^x, x taken into [-126, 127].
__device__ __forceinline__ float pow2i(int x) {
    return __int_as_float((min(max(x, -126), 127) + 127) << 23);
}

// Values that are not finite in a pair of 16 bits, and the pair without them.  kExp: the exponent
// bits.
constexpr uint32_t kExpBf16 = 0x7f80u, kExpF16 = 0x7c00u;
template <uint32_t kExp>
__device__ __forceinline__ bool not_finite2(uint32_t v) {
    return (v & kExp) == kExp || (v & (kExp << 16)) == (kExp << 16);
}
template <uint32_t kExp>
__device__ __forceinline__ uint32_t finite_part(uint32_t v) {
    if ((v & kExp) == kExp) v &= 0xffff0000u;
    if ((v & (kExp << 16)) == (kExp << 16)) v &= 0xffffu;
    return v;
}

// Page id of position p (0 <= p < max_pages * page_size) of sequence s, or -1 (reported)
// if the table holds none of the cache's pages there.
__device__ __forceinline__ int page_of(const tam_paged_batch& b, const tam_kv_cache& kv, int s,
                                       int page_shift, int p, int32_t* status, int kid) {
    const int id = b.page_table[(int64_t)s * b.max_pages + (p >> page_shift)];
    if ((uint32_t)id < (uint32_t)kv.n_pages) return id;
    report_error(status, TAM_ERR_PAGE, kid, s, p, id);
    return -1;
}

// Four e4m3 values -> fp32 (exact).
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float (&f)[4]) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

// 16 bytes of a cache row as fp32: 8 bf16, 4 fp32 or 16 e4m3 values.
template <int CD> struct CacheVec;
template <> struct CacheVec<TAM_F32> {
    static constexpr int N = 4, kBytes = 4;
    static __device__ __forceinline__ void to_f32(const uint4& w, float, float (&f)[4]) {
        f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y);
        f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
    }
};
template <> struct CacheVec<TAM_BF16> {
    static constexpr int N = 8, kBytes = 2;
    static __device__ __forceinline__ void to_f32(const uint4& w, float, float (&f)[8]) {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(x[i] << 16);
            f[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
        }
    }
};
template <> struct CacheVec<TAM_E4M3> {
    static constexpr int N = 16, kBytes = 1;
    static __device__ __forceinline__ void to_f32(const uint4& w, float scale, float (&f)[16]) {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y[4];
            e4m3x4_to_f32(x[i], y);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[4 * i + e] = y[e] * scale;   // exact: a power of two
        }
    }
};

}  // namespace tam

namespace tam {

// ---------------------------------------------------------------- work of a CTA
// The main kernels walk the (row block, KV head) items of the plan.  Dealt whole, CTA c
// takes the items c, c + grid, ...  Split, the units of all items stand in a row (block by
// block, head by head; `start` units for the item itself, then one per key tile) and CTA c
// takes the c-th of `grid` equal runs of them: the items whose tiles are all inside its run are
// its own, the ones at its two ends may be shared with its neighbours and leave a partial
// result in one of its two slots.
struct PagedItem {
    PagedBlock blk;
    int b, g;          // block, KV head
    int t0, t1;        // key tiles [t0, t1)
    int slot;          // partial slot to write (0, 1), or -1: the whole item is here
};

// a / b for 0 <= a, 0 < b: in 32 bits where a fits.
__device__ __forceinline__ int64_t div_small(int64_t a, int b) {
    return (a >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// The runs: the first `rest` CTAs take each + 1 units, the others `each`.
__device__ __forceinline__ int64_t run_start(const PagedPlan& p, int c) {
    return p.each * c + min(c, p.rest);
}
// The CTA whose run holds unit x.
__device__ __forceinline__ int run_of(const PagedPlan& p, int64_t x) {
    const int64_t longer = (p.each + 1) * p.rest;
    if ((x >> 31) == 0 && p.each < (1 << 30))
        return x < longer ? (int)((uint32_t)x / (uint32_t)(p.each + 1))
                          : p.rest + (int)((uint32_t)(x - longer) / (uint32_t)p.each);
    return x < longer ? (int)(x / (p.each + 1)) : p.rest + (int)((x - longer) / p.each);
}

// Chained launches: waits until the kernel before has finished and its writes are visible;
// lets the kernel after this one be launched.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename S>
__device__ __forceinline__ S ld_l2(const S* p) {
    static_assert(sizeof(S) % 8 == 0, "whole words");
    union { S s; long long w[sizeof(S) / 8]; } u;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(S) / 8); ++i) u.w[i] = __ldcg(reinterpret_cast<const long long*>(p) + i);
    return u.s;
}

// The block that holds unit x: the last one with unit0 * Hkv <= x.  32 candidates at a time,
// one per lane (by whole warps).
__device__ __forceinline__ int block_of(const PagedBlock* blocks, int n_blocks, int Hkv, int64_t x) {
    int l = 0, h = n_blocks - 1;
    const int lane = threadIdx.x & 31;
    while (l < h) {
        const int step = (h - l + 31) / 32;
        const int at = l + (lane + 1) * step;
        const bool below = at <= h && __ldcg(&blocks[at].unit0) * Hkv <= x;
        const int k = __popc(__ballot_sync(0xffffffffu, below));     // true for the first k
        l += k * step;
        h = min(h, l + step - 1);
    }
    return l;
}

struct PagedWalk {
    const PagedBlock* blocks;
    int Hkv, grid, start, b;
    bool whole;
    int64_t lo, pos, end;

    // by whole warps
    __device__ __forceinline__ PagedWalk(const PagedArgs& a, int cta)
        : blocks(a.blocks), Hkv(a.kv.Hkv), grid(a.grid), start(a.start) {
        const PagedPlan plan = *a.plan;
        const int n_blocks = plan.n_blocks;
        whole = plan.whole != 0;
        if (whole) {
            pos = cta;
            end = (int64_t)n_blocks * Hkv;
            return;
        }
        lo = pos = run_start(plan, cta);
        end = run_start(plan, cta + 1);
        b = block_of(blocks, n_blocks, Hkv, pos);
    }

    __device__ __forceinline__ bool next(PagedItem& it) {
        while (pos < end) {
            if (whole) {
                const int64_t blk = div_small(pos, Hkv);
                it.blk = blocks[blk];
                it.b = (int)blk;
                it.g = (int)(pos - blk * Hkv);
                it.t0 = 0;
                it.t1 = it.blk.nt;
                it.slot = -1;
                pos += grid;
                return true;
            }
            it.blk = blocks[b];
            it.b = b;
            const int units = start + it.blk.nt;
            const int64_t rel = pos - it.blk.unit0 * Hkv;
            it.g = (int)div_small(rel, units);
            const int u0 = (int)(rel - (int64_t)it.g * units);
            const int u1 = (int)min((int64_t)units, u0 + (end - pos));
            it.t0 = max(u0 - start, 0);
            it.t1 = max(u1 - start, 0);
            it.slot = (it.t0 == 0 && it.t1 == it.blk.nt) ? -1 : (pos == lo ? 0 : 1);
            pos += u1 - u0;
            if (u1 == units && it.g == Hkv - 1) ++b;
            if (it.t1 > it.t0) return true;            // else: its tiles are the next CTA's
        }
        return false;
    }
};

__device__ __forceinline__ float* part_slot(const PagedArgs& a, int cta, int slot) {
    return a.part + ((size_t)cta * 2 + slot) * paged_part_floats(a.rb, a.kv.d);
}

// Hands an item to the join's own computation, from whichever of its CTAs: its scales lie
// further apart than the products can take.
__device__ __forceinline__ void mark_redo(const PagedArgs& a, const PagedItem& it) {
    const int item = it.b * a.kv.Hkv + it.g;
    if (atomicExch(a.redo + kRedoMarks + item, 1) == 0)
        a.redo[kRedoMarks + a.redo_items + atomicAdd(a.redo, 1)] = item;
}

// log-sum-exp (natural) from a row's maximum (log2 domain) and sum; -inf for no key.
__device__ __forceinline__ float lse_of(float m, float l) {
    return l > 0.f || l != l ? m * kLn2 + logf(l) : -INFINITY;
}

}  // namespace tam
