// Attention over pages for a few rows per sequence (single tokens, drafted tokens).
//
//   x_j = scale*log2(e) * q.k_j,  out = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m)
//
// Bound: HBM.  Every K and V row is used by the 16 (or 32) rows of one block only, 4 bytes
// or less per multiply, so the tensor work is small and the point is to keep loads in
// flight.  The four warps of a CTA are independent: each streams its own keys (kKeys of
// every tile) through its own ring of shared-memory stages with cp.async, keeps its own
// running maximum, sum and output (mma.sync m16n8k16, bf16 operands, fp32 accumulators in
// registers) and meets the others only at the end of an item, where the four results are
// joined through shared memory.  No barrier runs per tile.  The 16 rows of a block are the
// query heads of the group times the new tokens, so every loaded row serves them all.
// 16 consecutive positions lie in one page (page_size >= 16), so a stage looks up one or
// two pages; the ids are fetched 32 at a time, one fetch ahead.
//
// Measured (device time of the three launches): 64 sequences of 100 to 8192 bf16 tokens, 32/8
// heads, d = 128 (1.05 GB) 182 us, 0.88 of the measured copy rate; 32 sequences of 1000 to 32768
// e4m3 tokens, 16/4 heads (0.51 GB) 112 us, 0.69, where half of the issue slots go to the
// instructions of the widened products; one sequence of 4096 tokens 16.5 us, three launches
// and their chains of dependent loads.
//
// e4m3: the bytes are widened to fp16 in registers (exact, one conversion per pair) and both
// products run on fp16 operands.  In the S product the order of the head dim is free as long
// as Q has the same one, so a thread takes 16 consecutive bytes of a K row as its operands of
// four k-steps; in the P V product the order of the columns of V is, so a thread takes D / 8
// consecutive bytes of each of its four V rows.  The scales stay out of the operands:
//   Q   is scaled by a power of two per row, its largest value to [2^14, 2^15): a bf16 value is
//       exact in fp16 then down to 2^-29 of the row's largest, and off by 2^-39 of it below;
//   K   2^e multiplies the scores (fp32, exact);
//   V   2^(e - E) goes into P before it is rounded, E the warp's reference exponent: O is kept
//       in units of 2^(E - kBase).  E follows the largest scale; a stage whose scales lie more
//       than 2^kSpread apart is taken in several passes, largest first, each with its own E,
//       so that no probability is lost to fp16's range: it keeps
//       11 bits (bf16 would keep 8) down to 2^-13 of the largest, and 2^-24 of it below that.
#include <algorithm>
#include <type_traits>

#include "launch.h"
#include "paged.cuh"
#include "tc_ptx.cuh"

namespace tam {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr float kLazy = 8.f;
constexpr int kBase = 7;              // e4m3: P is kept times 2^kBase, 2^15 with kLazy
constexpr uint32_t kSpread = 8;

template <int CD, int D, int MT>
struct Few {
    static constexpr bool kQuant = CD == TAM_E4M3;
    static constexpr int CB = CacheVec<CD>::kBytes;
    static constexpr int kRows = 16 * MT;
    // keys per warp and tile: 4 to 16 KB of K and V
    static constexpr int kKeys = (kQuant ? D <= 128 : D == 64) ? 32 : 16;
    static constexpr int kGroups = kKeys / 16;
    static constexpr int kRowBytes = D * CB;
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kTensor = kKeys * kRowBytes;             // one tensor's part of a stage
    static constexpr int kStage = 2 * kTensor + (kQuant ? 2 * kKeys : 0) + 16;
    // CTAs per SM: e4m3 is bound by instructions, not by bytes in flight, and wants warps (32
    // sequences of up to 32K tokens, d = 128: 132 us on two CTAs, 123 on three; four spill)
    static constexpr int kCtas = (2 * kTensor > 8192) ? 1 : (kQuant && MT * D <= 128) ? 3 : 2;
    static constexpr bool kQSmem = MT * D > 128 || kCtas > 2;     // else Q lives in registers
    static constexpr int kStages = (kCtas == 1 ? 192 : 200 / kCtas) * 1024 / (kWarps * 2 * kTensor);
    static constexpr int kQBytes = kQSmem ? kRows * D * 2 : 0;
    // XOR on the 16-byte column of a row of K (0) or V (1).  bf16: 8 rows of one column in 8
    // different bank groups (ldmatrix); e4m3: the 8 lanes of a quarter warp read 4 columns of 2
    // rows (K) or 2 columns of 4 rows (V)
    static constexpr __host__ __device__ int swizzle(int x, int row) {
        return !kQuant ? row & 7 : D == 64 ? 0 : x ? row & 6 : (row & 1) * 4;
    }
    static constexpr int kMergeLd = D + 8;
    static constexpr int kMerge = kWarps * kRows * (kMergeLd + 2) * 4;
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kSmem = kQBytes + (kRing > kMerge ? kRing : kMerge);
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
    // src-size 0 fills the 16 bytes with zeros and does not read src
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
// The low / high two e4m3 bytes of w -> fp16 pair (exact).
__device__ __forceinline__ uint32_t widen_lo(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// 2^x for -126 <= x <= 127
__device__ __forceinline__ float pow2i(int x) { return __int_as_float((x + 127) << 23); }
// Values that are not finite in a pair, and the pair without them.  kExp: the exponent bits.
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
constexpr uint32_t kExpBf16 = 0x7f80u, kExpF16 = 0x7c00u;

// e4m3: the column of V that thread group g (0..7) has as its n-th of D / 8, runs of up to
// 16 bytes of a row.
template <int D>
__device__ __forceinline__ int column_of(int g, int n) {
    if constexpr (D == 256) return (g + 8 * (n >> 4)) * 16 + (n & 15);
    else return g * (D / 8) + n;
}

template <int CD, int D, int MT>
__global__ void __launch_bounds__(kThreads, Few<CD, D, MT>::kCtas) k_paged_few(const PagedArgs a,
                                                                               int page_shift) {
    using F = Few<CD, D, MT>;
    constexpr bool kQuant = F::kQuant;
    constexpr int kKeys = F::kKeys, NT = kKeys / 8, NO = D / 8, KS = D / 16;
    extern __shared__ uint4 smem_raw4[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(smem_raw4);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t4 = lane & 3, g8 = lane >> 2;
    uint4* sq = reinterpret_cast<uint4*>(smem);                       // [MT][KS][32]
    uint8_t* ring = smem + F::kQBytes;
    const uint8_t* my_ring = ring + warp * F::kStages * F::kStage;
    const uint32_t mine = tc::smem_u32(my_ring);
    const int G = a.Hq / a.kv.Hkv, Hkv = a.kv.Hkv;
    const __nv_bfloat16* q = (const __nv_bfloat16*)a.q;

    wait_for_previous();                       // the plan
    let_next_start();                          // the join may read the plan while this runs
    PagedWalk walk(a, blockIdx.x);
    PagedItem it;
    while (walk.next(it)) {
        const PagedBlock& k = it.blk;
        const int n_rows = (int)min((int64_t)F::kRows, (int64_t)k.n * G - k.row0);
        // this thread's rows: g8 + 8 * i of the block
        int pos[2 * MT];
        const __nv_bfloat16* qrow[2 * MT];
        const int pos_min = k.pos0 + k.row0 / G;                      // of the block's first row
        const int pos_max = min(k.pos0 + (k.row0 + n_rows - 1) / G, k.len - 1);
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            const int r = g8 + 8 * i;
            const int row = k.row0 + r;
            pos[i] = r < n_rows ? k.pos0 + row / G : -1;
            qrow[i] = r < n_rows ? q + ((int64_t)(k.tok0 + row / G) * a.Hq + it.g * G + row % G) * D
                                 : nullptr;
        }
        // e4m3: the power of two on every row of Q, and its inverse times the score's scale
        float qs[2 * MT], fs[2 * MT];
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            qs[i] = 1.f;
            fs[i] = a.sl2;
            if constexpr (kQuant) {
                uint32_t top = 0;
                if (qrow[i])
#pragma unroll
                    for (int c = 0; c < D / 4; c += 8) {
                        const uint4 w = __ldg(reinterpret_cast<const uint4*>(qrow[i] + t4 * (D / 4) + c));
                        for (uint32_t x : {w.x, w.y, w.z, w.w})
                            top = max(top, max(x & 0x7fffu, (x >> 16) & 0x7fffu));
                    }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int sh = min(14 - ((int)(top >> 7) - 127), 120);
                qs[i] = pow2i(sh);
                fs[i] = a.sl2 * pow2i(-sh);
            }
        }
        // Q as A operands: registers 0..3 hold (row g8, k 2t..), (row g8+8, k 2t..), and the
        // same rows at k 2t+8..; `col` is where those k stand in the head dim
        uint32_t qf[F::kQSmem ? 1 : MT][F::kQSmem ? 1 : KS][4];
        auto q_frag = [&](int m, int kk, uint32_t (&r)[4]) {
            const int c0 = kQuant ? (t4 + 4 * (kk >> 2)) * 16 + (kk & 3) * 4 : kk * 16 + 2 * t4;
            const int c1 = kQuant ? c0 + 2 : c0 + 8;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const __nv_bfloat16* p = qrow[2 * m + i];
                r[i] = p ? __ldg(reinterpret_cast<const uint32_t*>(p + c0)) : 0u;
                r[2 + i] = p ? __ldg(reinterpret_cast<const uint32_t*>(p + c1)) : 0u;
                if constexpr (kQuant) {
                    r[i] = pack_f16(bf16_lo(r[i]) * qs[2 * m + i], bf16_hi(r[i]) * qs[2 * m + i]);
                    r[2 + i] = pack_f16(bf16_lo(r[2 + i]) * qs[2 * m + i],
                                        bf16_hi(r[2 + i]) * qs[2 * m + i]);
                }
            }
        };
        __syncthreads();                       // the last item's merge buffer is free
        if constexpr (F::kQSmem) {
            for (int x = warp; x < MT * KS; x += kWarps) {
                uint32_t r[4];
                // constant indices into qrow: m is 0 or 1
                if (MT == 1 || x < KS) q_frag(0, x, r);
                else q_frag(MT - 1, x - KS, r);
                sq[x * 32 + lane] = make_uint4(r[0], r[1], r[2], r[3]);
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) q_frag(m, kk, qf[m][kk]);
        }

        const int n_st = it.t1 - it.t0;
        const int first = it.t0 * (kWarps * kKeys) + warp * kKeys;    // first key of stage 0
        constexpr int kStep = kWarps * kKeys;
        // page ids of the next 32 / kGroups stages, one lane per 16 keys; -1: not there
        auto fetch_pages = [&](int u0) -> int {
            const int u = u0 + lane / F::kGroups;
            const int64_t j = (int64_t)first + (int64_t)u * kStep + (lane % F::kGroups) * 16;
            if (u >= n_st || j >= k.len) return -1;
            return page_of(a.b, a.kv, k.seq, page_shift, (int)j, a.status, KID_PAGED_FEW);
        };
        constexpr int kFetch = 32 / F::kGroups;
        int pages = fetch_pages(0), pages_next = fetch_pages(kFetch);
        // this lane's 16-byte column and first row of a 16-key group, and the step between rows
        constexpr int kPer = 16 * F::kChunks / 32, kRowStep = 32 / F::kChunks;   // copies per tensor
        const int ic = lane % F::kChunks, ir = lane / F::kChunks;
        const int64_t lane_off = (it.g * a.kv.head_stride + ir * a.kv.row_stride) * F::CB + ic * 16;
        const int64_t row_step = kRowStep * a.kv.row_stride * F::CB;
        const uint8_t* kp = (const uint8_t*)a.kv.k_pages + lane_off;
        const uint8_t* vp = (const uint8_t*)a.kv.v_pages + lane_off;
        // its place in a group: row ir, column ic, swizzled.  The swizzle is bitwise and y * kRowStep
        // and ir share no bits, so a row's swizzle is that of the two parts together
        const uint32_t lane_k = ir * F::kRowBytes + ((ic ^ F::swizzle(0, ir)) << 4);
        const uint32_t lane_v = ir * F::kRowBytes + ((ic ^ F::swizzle(1, ir)) << 4);
        int in_slot = 0;                        // ring slot of the next stage to be issued
        auto issue = [&](int u) {
            if (u < n_st) {
                if (u && u % kFetch == 0) {
                    pages = pages_next;
                    pages_next = fetch_pages(u + kFetch);
                }
                const uint32_t st = mine + in_slot * F::kStage;
                const int j0 = first + u * kStep;
#pragma unroll
                for (int h = 0; h < F::kGroups; ++h) {
                    const int page = __shfl_sync(0xffffffffu, pages, (u % kFetch) * F::kGroups + h);
                    const int in_page = (j0 + h * 16) & (a.kv.page_size - 1);
                    const int64_t off = ((int64_t)max(page, 0) * a.kv.page_stride +
                                         in_page * a.kv.row_stride) * F::CB;
                    // rows of this lane that are there: all, but behind the end of the sequence
                    const int rows = page < 0 ? 0 : k.len - (j0 + h * 16);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint8_t* src = (x ? vp : kp) + off;
#pragma unroll
                        for (int y = 0; y < kPer; ++y) {
                            const int r = y * kRowStep + ir;
                            const uint32_t dst = st + x * F::kTensor + (h * 16 + y * kRowStep) * F::kRowBytes +
                                                 ((x ? lane_v : lane_k) ^ (F::swizzle(x, y * kRowStep) << 4));
                            if (rows >= 16) cp_async16(dst, src + y * row_step);
                            else cp_async16(dst, src + y * row_step, r < rows);
                        }
                    }
                    if constexpr (kQuant) {
                        if (lane < 2) {                              // 16 scales of K and of V
                            const uint8_t* src = (lane ? a.kv.v_scale : a.kv.k_scale) +
                                (((int64_t)max(page, 0) * Hkv + it.g) << page_shift) + in_page;
                            cp_async16(st + 2 * F::kTensor + lane * kKeys + h * 16, src, page >= 0);
                        }
                    }
                    if (lane == 0) {
                        const uint32_t flag = st + 2 * F::kTensor + (kQuant ? 2 * kKeys : 0) + h * 4;
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(flag), "r"(page >= 0 ? 1 : 0) : "memory");
                    }
                }
                in_slot = in_slot + 1 == F::kStages ? 0 : in_slot + 1;
            }
            cp_commit();
        };

        float m[2 * MT], l[2 * MT], o[MT][NO][4];
        uint32_t ref_b = 0;                    // e4m3: the byte of E, 0 before the first key
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
#pragma unroll
        for (int x = 0; x < MT; ++x)
#pragma unroll
            for (int n = 0; n < NO; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[x][n][e] = 0.f;

#pragma unroll
        for (int u = 0; u < F::kStages - 1; ++u) issue(u);
        // e4m3: this thread's bytes of a stage: columns t4, t4 + 4, ... of the K row g8, and of the
        // V row 2 t4 the column g8 (g8 + 8 too for d = 256; a half of a column for d = 64)
        const uint32_t read_k = g8 * F::kRowBytes + ((t4 ^ F::swizzle(0, g8)) << 4);
        const uint32_t read_v = 2 * t4 * F::kRowBytes +
                                (D == 64 ? g8 * 8 : (g8 ^ F::swizzle(1, 2 * t4)) << 4);
        const int n_half = (n_rows + 7) / 8;   // halves of the row tiles that hold rows
        int slot = 0;
        for (int u = 0; u < n_st; ++u) {
            cp_wait<F::kStages - 2>();
            __syncwarp();                      // stage u is there, stage u - 1 is free
            issue(u + F::kStages - 1);
            const uint32_t st = mine + slot * F::kStage;
            const uint32_t sv = st + F::kTensor;
            // the same stage for plain loads (behind the wait's memory clobber)
            const uint8_t* gk = my_ring + slot * F::kStage;
            slot = slot + 1 == F::kStages ? 0 : slot + 1;
            const uint8_t* gv = gk + F::kTensor;
            const uint8_t* gsc = gk + 2 * F::kTensor;                 // e4m3: scales of K, then V
            const int j0 = first + u * kStep;

            // ---- S = Q K^T
            float s[MT][NT][4];
#pragma unroll
            for (int x = 0; x < MT; ++x)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[x][n][e] = 0.f;
            auto a_frag = [&](int x, int kk, uint32_t (&r)[4]) {
                if constexpr (F::kQSmem) {
                    const uint4 w = sq[(x * KS + kk) * 32 + lane];
                    r[0] = w.x; r[1] = w.y; r[2] = w.z; r[3] = w.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) r[e] = qf[x][kk][e];
                }
            };
            if constexpr (!kQuant) {
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    uint32_t af[MT][4];
#pragma unroll
                    for (int x = 0; x < MT; ++x) a_frag(x, kk, af[x]);
#pragma unroll
                    for (int h = 0; h < F::kGroups; ++h) {
                        const int row = h * 16 + (lane & 7) + (lane >> 4) * 8;
                        const int c = kk * 2 + ((lane >> 3) & 1);
                        uint32_t b[4];
                        ldsm4(b, st + row * F::kRowBytes + ((c ^ (row & 7)) << 4));
#pragma unroll
                        for (int x = 0; x < MT; ++x) {
                            mma(s[x][2 * h], af[x], b[0], b[1]);
                            mma(s[x][2 * h + 1], af[x], b[2], b[3]);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    uint4 w[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        w[n] = *reinterpret_cast<const uint4*>(gk + n * 8 * F::kRowBytes + (read_k ^ (i << 6)));
                    }
                    // k-step outside: the products of one column tile depend on one another
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        uint32_t af[MT][4];
#pragma unroll
                        for (int x = 0; x < MT; ++x) a_frag(x, 4 * i + y, af[x]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint32_t z = y == 0 ? w[n].x : y == 1 ? w[n].y : y == 2 ? w[n].z : w[n].w;
                            const uint32_t b0 = widen_lo(z), b1 = widen_hi(z);
#pragma unroll
                            for (int x = 0; x < MT; ++x) mma_f16(s[x][n], af[x], b0, b1);
                        }
                    }
                }
            }

            // ---- scale, mask, running maximum, P
            bool gone[F::kGroups];             // a group whose page is missing
            bool any_gone = false;
#pragma unroll
            for (int h = 0; h < F::kGroups; ++h) {
                const uint32_t f = *reinterpret_cast<const uint32_t*>(gsc + (kQuant ? 2 * kKeys : 0) + h * 4);
                gone[h] = f == 0;
                any_gone |= gone[h];
            }
            const bool cut = j0 + kKeys - 1 > pos_min;       // some row does not see some key
            float fk[kQuant ? NT : 1][2];
            if constexpr (kQuant) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint32_t two = *reinterpret_cast<const uint16_t*>(gsc + n * 8 + 2 * t4);
                    fk[n][0] = scale_value(two & 255u);
                    fk[n][1] = scale_value(two >> 8);
                }
            }
#pragma unroll
            for (int r = 0; r < 2 * MT; ++r) {
                float (&sr)[NT][4] = s[r >> 1];
                const int i2 = 2 * (r & 1);
                if (r >= n_half) {             // no rows: P = 0
#pragma unroll
                    for (int n = 0; n < NT; ++n) sr[n][i2] = sr[n][i2 + 1] = 0.f;
                    continue;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        sr[n][i2 + e] *= kQuant ? fk[kQuant ? n : 0][e] * fs[r] : fs[r];
                if (cut || any_gone) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (j0 + n * 8 + 2 * t4 + e > pos[r] || gone[n / 2]) sr[n][i2 + e] = -INFINITY;
                }
                float top = m[r];
#pragma unroll
                for (int n = 0; n < NT; ++n) top = tc::max3(top, sr[n][i2], sr[n][i2 + 1]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // raised lazily, so that O is rarely rescaled: P goes up to 2^kLazy
                const bool raise = top > m[r] + kLazy;
                const float ref = !raise ? (m[r] == -INFINITY ? 0.f : m[r]) : top;
                const float corr = raise ? tc::ex2(m[r] - top) : 1.f;
                float sum[2] = {0.f, 0.f};
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        sr[n][i2 + e] = tc::ex2(sr[n][i2 + e] - ref);
                        sum[e] += sr[n][i2 + e];
                    }
                l[r] = l[r] * corr + (sum[0] + sum[1]);
                if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                    for (int n = 0; n < NO; ++n) {
                        o[r >> 1][n][i2] *= corr;
                        o[r >> 1][n][i2 + 1] *= corr;
                    }
                }
                if (raise) m[r] = top;
            }

            // ---- O += P V.  Where some row does not see some key, what is not finite in V is
            // taken out of the product (0 times it is NaN) and added to the rows that see it.
            bool odd = false;
            auto clean = [&](uint32_t& b) {
                constexpr uint32_t kExp = kQuant ? kExpF16 : kExpBf16;
                odd |= not_finite2<kExp>(b);
                b = finite_part<kExp>(b);
            };
            if constexpr (!kQuant) {
                auto pv = [&](auto cut_tag) {
                    constexpr bool kCut = decltype(cut_tag)::value;
#pragma unroll
                    for (int h = 0; h < F::kGroups; ++h) {
                        uint32_t pf[MT][4];    // P rounded to bf16: the type of the product
#pragma unroll
                        for (int x = 0; x < MT; ++x) {
                            pf[x][0] = pack_bf16(s[x][2 * h][0], s[x][2 * h][1]);
                            pf[x][1] = pack_bf16(s[x][2 * h][2], s[x][2 * h][3]);
                            pf[x][2] = pack_bf16(s[x][2 * h + 1][0], s[x][2 * h + 1][1]);
                            pf[x][3] = pack_bf16(s[x][2 * h + 1][2], s[x][2 * h + 1][3]);
                        }
#pragma unroll
                        for (int n = 0; n < NO; n += 2) {
                            const int row = h * 16 + (lane & 15), c = n + (lane >> 4);
                            uint32_t b[4];
                            ldsm4t(b, sv + row * F::kRowBytes + ((c ^ (row & 7)) << 4));
                            if constexpr (kCut)
#pragma unroll
                                for (int e = 0; e < 4; ++e) clean(b[e]);
#pragma unroll
                            for (int x = 0; x < MT; ++x) {
                                mma(o[x][n], pf[x], b[0], b[1]);
                                mma(o[x][n + 1], pf[x], b[2], b[3]);
                            }
                        }
                    }
                };
                if (cut) pv(std::true_type{});
                else pv(std::false_type{});
            } else {
                float fv[F::kGroups][4];       // 2^(kBase + e - E) of this thread's keys
                auto pv = [&](auto careful_tag, bool nan_scale) {
                    constexpr bool kCareful = decltype(careful_tag)::value;
#pragma unroll
                    for (int h = 0; h < F::kGroups; ++h) {
                        uint32_t pf[MT][4];    // P rounded to fp16: the type of the product
#pragma unroll
                        for (int x = 0; x < MT; ++x) {
                            float y[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float p = s[x][2 * h + (e >> 2)][e & 3];
                                y[e] = p * fv[h][(e & 1) + (e >> 2) * 2];
                                if (kCareful && nan_scale && p == 0.f) y[e] = 0.f;
                            }
                            pf[x][0] = pack_f16(y[0], y[1]);
                            pf[x][1] = pack_f16(y[2], y[3]);
                            pf[x][2] = pack_f16(y[4], y[5]);
                            pf[x][3] = pack_f16(y[6], y[7]);
                        }
                        constexpr int RB = D / 8;                    // bytes per thread and row
                        constexpr int W = RB >= 16 ? 4 : 2;          // words per read
#pragma unroll
                        for (int z = 0; z < RB / (4 * W); ++z) {
                            uint32_t w[4][W];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint8_t* p = gv + (h * 16 + (e & 1) + (e >> 1) * 8) * F::kRowBytes + read_v;
                                if constexpr (W == 4) {
                                    const uint4 q4 = *reinterpret_cast<const uint4*>(p + z * 128);
                                    w[e][0] = q4.x; w[e][1] = q4.y; w[e][2] = q4.z; w[e][3] = q4.w;
                                } else {
                                    const uint2 q2 = *reinterpret_cast<const uint2*>(p);
                                    w[e][0] = q2.x; w[e][1] = q2.y;
                                }
                            }
#pragma unroll
                            for (int v = 0; v < W; ++v)
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    // bytes 2y, 2y + 1 of two rows: two pairs over the keys
                                    const uint32_t sel = y ? 0x7362 : 0x5140;
                                    const uint32_t u0 = __byte_perm(w[0][v], w[1][v], sel);
                                    const uint32_t u1 = __byte_perm(w[2][v], w[3][v], sel);
                                    uint32_t b[4] = {widen_lo(u0), widen_lo(u1), widen_hi(u0), widen_hi(u1)};
                                    if constexpr (kCareful)
#pragma unroll
                                        for (int e = 0; e < 4; ++e) clean(b[e]);
                                    const int n = z * 4 * W + v * 4 + y * 2;
#pragma unroll
                                    for (int x = 0; x < MT; ++x) {
                                        mma_f16(o[x][n], pf[x], b[0], b[1]);
                                        mma_f16(o[x][n + 1], pf[x], b[2], b[3]);
                                    }
                                }
                        }
                    }
                };
                // the scales of the keys some row sees: one lane per key; 0 = none, 255 = NaN
                uint32_t byte = 0;
                if (lane < kKeys && j0 + lane <= pos_max) byte = gsc[kKeys + lane];
                // all of them at most 2^kSpread below the reference, every key seen: the common case
                const bool plain = !cut && !any_gone &&
                                   __all_sync(0xffffffffu, lane >= kKeys || (byte && ref_b - byte <= kSpread));
                if (plain) {
                    const uint32_t base = (127u + kBase - ref_b) << 23;
#pragma unroll
                    for (int h = 0; h < F::kGroups; ++h)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t two = *reinterpret_cast<const uint16_t*>(
                                gsc + kKeys + h * 16 + 2 * t4 + e * 8);
                            fv[h][2 * e] = __uint_as_float(((two & 255u) << 23) + base);
                            fv[h][2 * e + 1] = __uint_as_float((two >> 8 << 23) + base);
                        }
                    pv(std::false_type{}, false);
                } else {
                    const bool nan_scale = __any_sync(0xffffffffu, byte == kScaleNan);
                    const uint32_t seen = byte == kScaleNan ? 0u : byte;
                    uint32_t below = 255;      // this pass takes the scales below this
                    do {
                        const uint32_t mine_b = seen < below ? seen : 0u;
                        const uint32_t top = __reduce_max_sync(0xffffffffu, mine_b);
                        const uint32_t low = __reduce_min_sync(0xffffffffu, mine_b ? mine_b : 255u);
                        // keep the reference while it serves: within kSpread above every scale
                        if (top > ref_b || (top && low + kSpread < ref_b)) {
                            if (ref_b) {
                                const int d = (int)ref_b - (int)top;         // exact: powers of two
                                const float f = pow2i(min(max(d / 2, -126), 127));
                                const float f2 = pow2i(min(max(d - d / 2, -126), 127));
#pragma unroll
                                for (int x = 0; x < MT; ++x)
#pragma unroll
                                    for (int n = 0; n < NO; ++n)
#pragma unroll
                                        for (int e = 0; e < 4; ++e) o[x][n][e] = o[x][n][e] * f * f2;
                            }
                            ref_b = top;
                        }
                        const uint32_t from = ref_b > kSpread ? ref_b - kSpread : 0u;   // this pass
#pragma unroll
                        for (int h = 0; h < F::kGroups; ++h)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t bb = __shfl_sync(0xffffffffu, byte,
                                                                h * 16 + 2 * t4 + (e & 1) + (e >> 1) * 8);
                                fv[h][e] = bb >= from && bb < below && bb != 0u
                                               ? __uint_as_float((bb + 127u + kBase - ref_b) << 23) : 0.f;
                                if (bb == kScaleNan) fv[h][e] = __int_as_float(0x7fc00000);
                            }
                        pv(std::true_type{}, nan_scale);
                        below = from;
                    } while (__any_sync(0xffffffffu, seen != 0u && seen < below));
                }
            }
            if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
                for (int j = 0; j < kKeys; ++j) {
#pragma unroll
                    for (int n = 0; n < NO; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float v;
                            if constexpr (kQuant) {
                                const int dim = column_of<D>(2 * t4 + e, n);
                                const uint8_t w = gv[j * F::kRowBytes + (((dim >> 4) ^ F::swizzle(1, j)) << 4) + (dim & 15)];
                                float f[4];
                                e4m3x4_to_f32(w, f);
                                v = f[0];      // a NaN scale came with P
                            } else {
                                const int dim = n * 8 + 2 * t4 + e;
                                v = to_f(*reinterpret_cast<const __nv_bfloat16*>(
                                    gv + j * F::kRowBytes + (((dim >> 3) ^ (j & 7)) << 4) + (dim & 7) * 2));
                            }
                            if (isfinite(v)) continue;
#pragma unroll
                            for (int r = 0; r < 2 * MT; ++r)
                                if (j0 + j <= pos[r]) o[r >> 1][n][2 * (r & 1) + e] += v;
                        }
                }
            }
        }
        cp_wait<0>();

        // ---- join the four warps
        if constexpr (kQuant) {
            const float unit = ref_b ? pow2i(max((int)ref_b - 127 - kBase, -126)) : 0.f;
#pragma unroll
            for (int x = 0; x < MT; ++x)
#pragma unroll
                for (int n = 0; n < NO; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[x][n][e] *= unit;
        }
#pragma unroll
        for (int r = 0; r < 2 * MT; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        }
        __syncthreads();                       // every warp has left its ring
        float* mo = reinterpret_cast<float*>(ring);                  // [warp][row][kMergeLd]
        float* mm = mo + kWarps * F::kRows * F::kMergeLd;            // [warp][row] maxima
        float* ml = mm + kWarps * F::kRows;                          // sums
#pragma unroll
        for (int r = 0; r < 2 * MT; ++r) {
            const int row = g8 + 8 * r;
            float* d = mo + (warp * F::kRows + row) * F::kMergeLd;
#pragma unroll
            for (int n = 0; n < NO; ++n) {
                const float x = o[r >> 1][n][2 * (r & 1)], y = o[r >> 1][n][2 * (r & 1) + 1];
                if constexpr (kQuant) {
                    d[column_of<D>(2 * t4, n)] = x;
                    d[column_of<D>(2 * t4 + 1, n)] = y;
                } else {
                    *reinterpret_cast<float2*>(d + n * 8 + 2 * t4) = make_float2(x, y);
                }
            }
            if (t4 == 0) {
                mm[warp * F::kRows + row] = m[r];
                ml[warp * F::kRows + row] = l[r];
            }
        }
        __syncthreads();
        constexpr int kLanes = kThreads / 16;                         // threads per row
#pragma unroll
        for (int r0 = 0; r0 < F::kRows; r0 += 16) {
            const int r = r0 + threadIdx.x / kLanes, c0 = (threadIdx.x % kLanes) * 4;
            if (r >= n_rows) continue;
            float M = -INFINITY, f[kWarps], sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mm[w * F::kRows + r]);
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                f[w] = tc::ex2(mm[w * F::kRows + r] - ref);
                sum += f[w] * ml[w * F::kRows + r];
            }
            const bool part = it.slot >= 0;
            float* ps = part ? part_slot(a, blockIdx.x, it.slot) : nullptr;
            const float inv = part ? 1.f : (sum > 0.f || sum != sum ? 1.f / sum : 0.f);
            const int row = k.row0 + r;
            const int64_t tok = k.tok0 + row / G;
            const int head = it.g * G + row % G;
#pragma unroll
            for (int c = 0; c < D; c += kLanes * 4) {
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 z = *reinterpret_cast<const float4*>(
                        mo + (w * F::kRows + r) * F::kMergeLd + c + c0);
                    y.x += f[w] * z.x; y.y += f[w] * z.y; y.z += f[w] * z.z; y.w += f[w] * z.w;
                }
                if (part)
                    *reinterpret_cast<float4*>(ps + (size_t)r * D + c + c0) = y;
                else
                    *reinterpret_cast<uint2*>((__nv_bfloat16*)a.out + (tok * a.Hq + head) * D + c + c0) =
                        make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
            }
            if (c0 == 0) {
                if (part) {
                    ps[(size_t)F::kRows * D + r] = M;
                    ps[(size_t)F::kRows * (D + 1) + r] = sum;
                } else if (a.lse) {
                    a.lse[(int64_t)a.Hq * k.tok0 + (int64_t)head * k.n + row / G] = lse_of(M, sum);
                }
            }
        }
    }
}

template <int CD, int D, int MT>
cudaError_t launch(const PagedArgs& a, cudaStream_t st) {
    using F = Few<CD, D, MT>;
    static_assert(F::kSmem <= 227 * 1024 / F::kCtas - 1024, "stages exceed shared memory");
    auto kern = k_paged_few<CD, D, MT>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem((const void*)kern, F::kSmem, done);
    if (e != cudaSuccess) return e;
    int shift = 0;
    while ((1 << shift) < a.kv.page_size) ++shift;
    if ((e = launch_chained(kern, a.grid, kThreads, F::kSmem, st, a, shift))) return e;
    note_launch();
    return cudaSuccess;
}

// Applies fn.template operator()<CD, D, MT>() for the call's shape.
template <class Fn>
auto by_shape(const PagedArgs& a, Fn fn) {
    const bool two = (int64_t)a.b.max_rows * (a.Hq / a.kv.Hkv) > 16 && a.kv.d <= 128;
    const bool quant = a.kv.dtype == TAM_E4M3;
    switch (a.kv.d) {
        case 64:
            if (two) return quant ? fn.template operator()<TAM_E4M3, 64, 2>() : fn.template operator()<TAM_BF16, 64, 2>();
            return quant ? fn.template operator()<TAM_E4M3, 64, 1>() : fn.template operator()<TAM_BF16, 64, 1>();
        case 128:
            if (two) return quant ? fn.template operator()<TAM_E4M3, 128, 2>() : fn.template operator()<TAM_BF16, 128, 2>();
            return quant ? fn.template operator()<TAM_E4M3, 128, 1>() : fn.template operator()<TAM_BF16, 128, 1>();
        default:
            return quant ? fn.template operator()<TAM_E4M3, 256, 1>() : fn.template operator()<TAM_BF16, 256, 1>();
    }
}

// An item's own cost (Q, the first loads, the join of the warps), in tiles.
constexpr int kStart = 4;
struct ShapeOf {
    template <int CD, int D, int MT>
    PagedShape operator()() const {
        using F = Few<CD, D, MT>;
        return {F::kRows, kWarps * F::kKeys, 148 * F::kCtas, kStart};
    }
};
struct Launch {
    const PagedArgs& a;
    cudaStream_t st;
    template <int CD, int D, int MT>
    cudaError_t operator()() const { return launch<CD, D, MT>(a, st); }
};

}  // namespace

bool paged_few_supported(const PagedArgs& a) {
    const int64_t rows = (int64_t)a.b.max_rows * (a.Hq / a.kv.Hkv);
    return a.dtype == TAM_BF16 && rows > 0 && rows <= (a.kv.d <= 128 ? 32 : 16);
}

PagedShape paged_few_shape(const PagedArgs& a) { return by_shape(a, ShapeOf{}); }

cudaError_t paged_few(const PagedArgs& a, cudaStream_t st) { return by_shape(a, Launch{a, st}); }

}  // namespace tam
