// Attention over pages for a few rows per sequence (single tokens, drafted tokens).
//
//   x_j = scale*log2(e) * q.k_j,  out = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m)
//
// Bound: HBM.  Every K and V row is used by the 8 to 32 rows of one block only, 8 bytes or
// less per multiply, so the tensor work is small and the point is to keep loads in flight.
// The four warps of a CTA are independent: each streams its own keys (kKeys of every tile)
// through its own ring of shared-memory stages with cp.async, keeps its own running maximum,
// sum and output and meets the others only at the end of an item, where the four results are
// joined through shared memory.  No barrier runs per tile.  The rows of a block are the query
// heads of the group times the new tokens, so every loaded row serves them all.  16
// consecutive positions lie in one page (page_size >= 16), so a stage looks up one or two
// pages; the ids are fetched 32 at a time, one fetch ahead.
//
// The products are taken transposed, S^T = K Q^T and O^T += V^T P^T, by mma.sync m16n8k16 with
// fp32 accumulators in registers: the cache fills the 16 rows of the instruction and the few
// rows of a block its 8 columns, so a block has RT = 1 to 4 tiles of 8 rows and a group of
// four query heads fills half of a product and not a quarter.  P leaves S^T with the keys down
// the lanes and enters the second product with the rows there: one 8x8 transpose per operand
// register.  (32 sequences of up to 32K e4m3 tokens, 16/4 heads, d = 128: 102 us so, 111 with
// the rows of Q as the 16 rows; 20 rows of 16 sequences, d = 64: 39 us, 45.)  The running maximum
// is raised only when a score is 2^kLazy above it, so a stage asks one vote and no reduction.
//
// Measured (device time of the three launches, behind a read of 320 MB): 64 sequences of 100 to 8192
// bf16 tokens, 32/8 heads, d = 128 (1.05 GB) 181 us, 0.88 of the measured copy rate; 32 sequences of
// 1000 to 32768 e4m3 tokens, 16/4 heads (0.51 GB) 104 us, 0.74, and 127 us with 16 rows per KV head,
// where the instructions that widen the cache take the issue slots; one sequence of 4096 bf16 tokens
// 17 us (14 with the cache in L2), three launches and their chains of dependent loads.  Some 12 us of
// each are the plan, the first loads of the items and the joins.  (The figures beside the choices
// below and in the code were taken while each was made, call after call, and compare with one
// another.)
//
// e4m3: the bytes are widened to fp16 in registers (exact, one conversion per pair) and both
// products run on fp16 operands.  (The S product on the e4m3 bytes themselves, Q split into two
// e4m3 parts, took 146 us where this took 111: the 8-bit mma.sync has no higher rate here.)  In
// the S product the order of the head dim is free as long as Q has the same one, so a thread
// takes 16 consecutive bytes of a K row as its operands of four k-steps; V is transposed by the
// byte form of ldmatrix, which hands a lane four consecutive keys of a column, two pairs of one
// k-step: the keys of S^T are taken in that order.  (With bytes of two rows paired by byte
// permutes instead, 16 rows of d = 128 took 135 us and not 125.)  The scales stay out of the
// operands:
//   Q   is scaled by a power of two per row, its largest value to [2^14, 2^15): a bf16 value is
//       exact in fp16 then down to 2^-29 of the row's largest, and off by 2^-39 of it below;
//   K   2^e multiplies the scores (fp32, exact);
//   V   2^(e - E) goes into P before it is rounded, E the warp's reference exponent: O is kept
//       in units of 2^(E - kBase).  E follows the largest scale; a stage whose scales lie more
//       than 2^kSpread apart is taken in several passes, largest first, each with its own E,
//       so that no probability is lost to fp16's range: it keeps
//       11 bits (bf16 would keep 8) down to 2^-13 of the largest, and 2^-24 of it below that.
//       An item whose scales span more than 2^kSpan is computed again by the join (what small
//       probabilities of the largest rows add would lose its bits, and O overflow on the way
//       down); rows of zeros do not count.
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

template <int CD, int D, int RT>
struct Few {
    static constexpr bool kQuant = CD == TAM_E4M3;
    static constexpr int CB = CacheVec<CD>::kBytes;
    static constexpr int kRows = 8 * RT;
    // keys per warp and tile: 4 to 16 KB of K and V
    static constexpr int kKeys = (kQuant ? D <= 128 : D == 64) ? 32 : 16;
    static constexpr int kGroups = kKeys / 16;
    static constexpr int kRowBytes = D * CB;
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kTensor = kKeys * kRowBytes;             // one tensor's part of a stage
    static constexpr int kStage = 2 * kTensor + (kQuant ? 2 * kKeys : 0) + 16;
    // CTAs per SM: e4m3 is bound by latencies and instructions and wants warps, as long as the
    // registers do (d = 64: 24 rows take 39 us on three, 40 on two, 51 on four CTAs, 32 rows 237
    // on three, which spills, and 144 on two; d = 256, 8 rows 117 on three, 108 on two)
    static constexpr int kCtas = (2 * kTensor > 8192) ? 1 : (kQuant && RT * D <= 192) ? 3 : 2;
    static constexpr bool kQSmem = RT * D > 256 || kCtas > 2;     // else Q lives in registers
    static constexpr int kStages = (kCtas == 1 ? 192 : 200 / kCtas) * 1024 / (kWarps * 2 * kTensor);
    static constexpr int kQBytes = kQSmem ? kRows * D * 2 : 0;
    // XOR on the 16-byte column of a row of K (0) or V (1).  bf16: 8 rows of one column in 8
    // different bank groups (ldmatrix), and so for V of e4m3; of its K, the 8 lanes of a quarter
    // warp read 4 columns of 2 rows
    static constexpr __host__ __device__ int swizzle(int x, int row) {
        return !kQuant ? row & 7 : x ? (D == 64 ? row >> 1 & 3 : row & 7) : D == 64 ? 0 : (row & 1) * 4;
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
// Two 16x16 matrices of bytes, transposed: lane 4 i + j gets of the columns i, i + 8 of the first,
// then of the second, the rows 4 j .. 4 j + 3.  Lane l gives the address of row l % 16 of matrix
// l / 16.
__device__ __forceinline__ void ldsm_bytes(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
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
// A transposed 8x8 matrix of 16-bit elements: lane 4 i + j holds (i, 2 j) and (i, 2 j + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
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

template <int CD, int D, int RT>
__global__ void __launch_bounds__(kThreads, Few<CD, D, RT>::kCtas) k_paged_few(const PagedArgs a,
                                                                               int page_shift) {
    using F = Few<CD, D, RT>;
    constexpr bool kQuant = F::kQuant;
    constexpr int kKeys = F::kKeys, H = F::kGroups, NO = D / 16, KS = D / 16;
    extern __shared__ uint4 smem_raw4[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(smem_raw4);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t4 = lane & 3, g8 = lane >> 2;
    uint2* sq = reinterpret_cast<uint2*>(smem);                       // [RT][KS][32]
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
        const int pos_min = k.pos0 + k.row0 / G;                      // of the block's first row
        const int pos_max = min(k.pos0 + (k.row0 + n_rows - 1) / G, k.len - 1);
        // this thread's scores are of the rows 8 * x + 2 * t4 + e; it loads Q's rows 8 * x + g8
        int pos[2 * RT];
        const __nv_bfloat16* qrow[RT];
#pragma unroll
        for (int i = 0; i < 2 * RT; ++i) {
            const int r = 8 * (i >> 1) + 2 * t4 + (i & 1);
            pos[i] = r < n_rows ? k.pos0 + (k.row0 + r) / G : -1;
        }
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            const int r = 8 * x + g8;
            const int row = k.row0 + r;
            qrow[x] = r < n_rows ? q + ((int64_t)(k.tok0 + row / G) * a.Hq + it.g * G + row % G) * D
                                 : nullptr;
        }
        // e4m3: the power of two on every row of Q, and its inverse times the score's scale
        float qs[RT], fs[2 * RT];
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            qs[x] = 1.f;
            fs[2 * x] = fs[2 * x + 1] = a.sl2;
            if constexpr (kQuant) {
                uint32_t top = 0;
                if (qrow[x])
#pragma unroll
                    for (int c = 0; c < D / 4; c += 8) {
                        const uint4 w = __ldg(reinterpret_cast<const uint4*>(qrow[x] + t4 * (D / 4) + c));
                        for (uint32_t v : {w.x, w.y, w.z, w.w})
                            top = max(top, max(v & 0x7fffu, (v >> 16) & 0x7fffu));
                    }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int sh = min(14 - ((int)(top >> 7) - 127), 120);
                qs[x] = pow2i(sh);
                const float f = a.sl2 * pow2i(-sh);
#pragma unroll
                for (int e = 0; e < 2; ++e) fs[2 * x + e] = __shfl_sync(0xffffffffu, f, (2 * t4 + e) * 4);
            }
        }
        // Q as B operands: registers 0 and 1 hold row g8 at k 2t.. and 2t+8..; `col` is where
        // those k stand in the head dim
        uint32_t qf[F::kQSmem ? 1 : RT][F::kQSmem ? 1 : KS][2];
        auto q_frag = [&](const __nv_bfloat16* p, float f, int kk, uint32_t (&r)[2]) {
            const int col = kQuant ? (t4 + 4 * (kk >> 2)) * 16 + (kk & 3) * 4 : kk * 16 + 2 * t4;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                r[i] = p ? __ldg(reinterpret_cast<const uint32_t*>(p + col + i * (kQuant ? 2 : 8))) : 0u;
                if constexpr (kQuant) r[i] = pack_f16(bf16_lo(r[i]) * f, bf16_hi(r[i]) * f);
            }
        };
        __syncthreads();                       // the last item's merge buffer is free
        if constexpr (F::kQSmem) {
#pragma unroll
            for (int x = 0; x < RT; ++x)
                for (int kk = warp; kk < KS; kk += kWarps) {
                    uint32_t r[2];
                    q_frag(qrow[x], qs[x], kk, r);
                    sq[(x * KS + kk) * 32 + lane] = make_uint2(r[0], r[1]);
                }
            __syncthreads();
        } else {
#pragma unroll
            for (int x = 0; x < RT; ++x)
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) q_frag(qrow[x], qs[x], kk, qf[x][kk]);
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
                for (int h = 0; h < H; ++h) {
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

        // o[x][n]: the columns 16 n + g8 (registers 0, 1) and 16 n + 8 + g8 (2, 3), rows
        // 8 * x + 2 * t4 + {0, 1}
        float m[2 * RT], l[2 * RT], o[RT][NO][4];
        uint32_t ref_b = 0;                    // e4m3: the byte of E, 0 before the first key
        uint32_t ref_high = 0;                 // its largest value
        uint32_t low_b = 255;                  // this lane's smallest scale byte, less one
#pragma unroll
        for (int i = 0; i < 2 * RT; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
#pragma unroll
        for (int x = 0; x < RT; ++x)
#pragma unroll
            for (int n = 0; n < NO; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[x][n][e] = 0.f;

#pragma unroll
        for (int u = 0; u < F::kStages - 1; ++u) issue(u);
        // This thread's keys in a group of 16: key0 (registers 0, 1 of s) and key0 + key_step (2, 3).
        // e4m3: the order in which the transposed load of V hands the keys over
        const int key0 = kQuant ? (g8 >> 1) * 4 + (g8 & 1) : g8;
        constexpr int key_step = kQuant ? 2 : 8;
        // e4m3: this thread's bytes of K: columns t4, t4 + 4, ... of the row key0; and its row and
        // column of V for the transposed load
        const uint32_t read_k = key0 * F::kRowBytes + ((t4 ^ F::swizzle(0, key0)) << 4);
        const uint32_t read_v = (lane & 15) * F::kRowBytes + (((lane >> 4) ^ F::swizzle(1, lane & 15)) << 4);
        const int n_tile = (n_rows + 7) / 8;   // row tiles that hold rows
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

            // ---- S^T = K Q^T: s[x][h]: keys of the group h
            float s[RT][H][4];
#pragma unroll
            for (int x = 0; x < RT; ++x)
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[x][h][e] = 0.f;
            auto b_frag = [&](int x, int kk, uint32_t (&r)[2]) {
                if constexpr (F::kQSmem) {
                    const uint2 w = sq[(x * KS + kk) * 32 + lane];
                    r[0] = w.x; r[1] = w.y;
                } else {
                    r[0] = qf[x][kk][0]; r[1] = qf[x][kk][1];
                }
            };
            if constexpr (!kQuant) {
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    uint32_t bf[RT][2];
#pragma unroll
                    for (int x = 0; x < RT; ++x) b_frag(x, kk, bf[x]);
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        const int row = h * 16 + (lane & 15);
                        const int c = kk * 2 + (lane >> 4);
                        uint32_t af[4];
                        ldsm4(af, st + row * F::kRowBytes + ((c ^ (row & 7)) << 4));
#pragma unroll
                        for (int x = 0; x < RT; ++x) mma(s[x][h], af, bf[x][0], bf[x][1]);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    uint4 w[2 * H];
#pragma unroll
                    for (int n = 0; n < 2 * H; ++n)
                        w[n] = *reinterpret_cast<const uint4*>(gk + ((n >> 1) * 16 + (n & 1) * key_step) * F::kRowBytes + (read_k ^ (i << 6)));
                    // k-step outside: the products of one group depend on one another
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        uint32_t bf[RT][2];
#pragma unroll
                        for (int x = 0; x < RT; ++x) b_frag(x, 4 * i + y, bf[x]);
                        auto word = [&](const uint4& v) { return y == 0 ? v.x : y == 1 ? v.y : y == 2 ? v.z : v.w; };
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            const uint32_t z0 = word(w[2 * h]), z1 = word(w[2 * h + 1]);
                            const uint32_t af[4] = {widen_lo(z0), widen_lo(z1), widen_hi(z0), widen_hi(z1)};
#pragma unroll
                            for (int x = 0; x < RT; ++x) mma_f16(s[x][h], af, bf[x][0], bf[x][1]);
                        }
                    }
                }
            }

            // ---- scale, mask, running maximum, P
            bool gone[H];                      // a group whose page is missing
            bool any_gone = false;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const uint32_t f = *reinterpret_cast<const uint32_t*>(gsc + (kQuant ? 2 * kKeys : 0) + h * 4);
                gone[h] = f == 0;
                any_gone |= gone[h];
            }
            const bool cut = j0 + kKeys - 1 > pos_min;       // some row does not see some key
            float fk[kQuant ? H : 1][2];
            if constexpr (kQuant) {
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i) fk[h][i] = scale_value(gsc[h * 16 + i * key_step + key0]);
            }
#pragma unroll
            for (int x = 0; x < RT; ++x) {
                if (x >= n_tile) {             // no rows: P = 0
#pragma unroll
                    for (int h = 0; h < H; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[x][h][e] = 0.f;
                    continue;
                }
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[x][h][e] *= kQuant ? fk[kQuant ? h : 0][e >> 1] * fs[2 * x + (e & 1)] : fs[2 * x + (e & 1)];
                if (cut || any_gone) {
#pragma unroll
                    for (int h = 0; h < H; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (j0 + h * 16 + key0 + (e >> 1) * key_step > pos[2 * x + (e & 1)] || gone[h])
                                s[x][h][e] = -INFINITY;
                }
                // the maximum is raised lazily, so that O is rarely rescaled: P goes up to 2^kLazy
                float top[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[e] = m[2 * x + e];
#pragma unroll
                    for (int h = 0; h < H; ++h) top[e] = tc::max3(top[e], s[x][h][e], s[x][h][2 + e]);
                }
                if (__any_sync(0xffffffffu, top[0] > m[2 * x] + kLazy || top[1] > m[2 * x + 1] + kLazy)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float& mr = m[2 * x + e];
#pragma unroll
                        for (int d = 4; d < 32; d *= 2)
                            top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], d));
                        const bool raise = top[e] > mr + kLazy;
                        const float corr = raise ? tc::ex2(mr - top[e]) : 1.f;
                        l[2 * x + e] *= corr;
#pragma unroll
                        for (int n = 0; n < NO; ++n) {
                            o[x][n][e] *= corr;
                            o[x][n][2 + e] *= corr;
                        }
                        if (raise) mr = top[e];
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float ref = m[2 * x + e] == -INFINITY ? 0.f : m[2 * x + e];
                    float sum[2] = {0.f, 0.f};
#pragma unroll
                    for (int h = 0; h < H; ++h)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            s[x][h][2 * i + e] = tc::ex2(s[x][h][2 * i + e] - ref);
                            sum[i] += s[x][h][2 * i + e];
                        }
                    l[2 * x + e] += sum[0] + sum[1];
                }
            }

            // ---- O^T += V^T P^T.  Where some row does not see some key, what is not finite in V is
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
                    for (int h = 0; h < H; ++h) {
                        uint32_t pf[RT][2];    // P rounded to bf16: the type of the product
#pragma unroll
                        for (int x = 0; x < RT; ++x)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                pf[x][i] = transpose8(pack_bf16(s[x][h][2 * i], s[x][h][2 * i + 1]));
#pragma unroll
                        for (int n = 0; n < NO; ++n) {
                            const int row = h * 16 + (lane & 7) + (lane >> 4) * 8;
                            const int c = 2 * n + ((lane >> 3) & 1);
                            uint32_t af[4];
                            ldsm4t(af, sv + row * F::kRowBytes + ((c ^ (row & 7)) << 4));
                            if constexpr (kCut)
#pragma unroll
                                for (int e = 0; e < 4; ++e) clean(af[e]);
#pragma unroll
                            for (int x = 0; x < RT; ++x) mma(o[x][n], af, pf[x][0], pf[x][1]);
                        }
                    }
                };
                if (cut) pv(std::true_type{});
                else pv(std::false_type{});
            } else {
                float fv[H][2];                // 2^(kBase + e - E) of this thread's keys
                auto pv = [&](auto careful_tag, bool nan_scale) {
                    constexpr bool kCareful = decltype(careful_tag)::value;
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        uint32_t pf[RT][2];    // P rounded to fp16: the type of the product
#pragma unroll
                        for (int x = 0; x < RT; ++x)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                float y[2];
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const float p = s[x][h][2 * i + e];
                                    y[e] = p * fv[h][i];
                                    if (kCareful && nan_scale && p == 0.f) y[e] = 0.f;
                                }
                                pf[x][i] = transpose8(pack_f16(y[0], y[1]));
                            }
#pragma unroll
                        for (int z = 0; z < D / 32; ++z) {
                            uint32_t w[4];
                            ldsm_bytes(w, sv + h * 16 * F::kRowBytes + (read_v ^ (z << 5)));
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                uint32_t af[4] = {widen_lo(w[2 * y]), widen_lo(w[2 * y + 1]),
                                                  widen_hi(w[2 * y]), widen_hi(w[2 * y + 1])};
                                if constexpr (kCareful)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) clean(af[e]);
#pragma unroll
                                for (int x = 0; x < RT; ++x) mma_f16(o[x][2 * z + y], af, pf[x][0], pf[x][1]);
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
                    low_b = min(low_b, byte - 1);
                    const uint32_t base = (127u + kBase - ref_b) << 23;
#pragma unroll
                    for (int h = 0; h < H; ++h)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            fv[h][i] = __uint_as_float(((uint32_t)gsc[kKeys + h * 16 + i * key_step + key0] << 23) + base);
                    pv(std::false_type{}, false);
                } else {
                    if (__any_sync(0xffffffffu, byte && byte <= kScaleLeast)) {
                        uint32_t any = 0;      // a row of zeros needs no scale
                        if (byte && byte <= kScaleLeast)
                            for (int c = 0; c < F::kChunks; ++c) {
                                const uint4 w = *reinterpret_cast<const uint4*>(gv + lane * F::kRowBytes + c * 16);
                                any |= (w.x | w.y | w.z | w.w) & 0x7f7f7f7fu;
                            }
                        if (byte <= kScaleLeast && !any) byte = 0;
                    }
                    const bool nan_scale = __any_sync(0xffffffffu, byte == kScaleNan);
                    const uint32_t seen = byte == kScaleNan ? 0u : byte;
                    low_b = min(low_b, seen - 1);
                    uint32_t below = 255;      // this pass takes the scales below this
                    do {
                        const uint32_t mine_b = seen < below ? seen : 0u;
                        const uint32_t top = __reduce_max_sync(0xffffffffu, mine_b);
                        const uint32_t low = __reduce_min_sync(0xffffffffu, mine_b ? mine_b : 255u);
                        // keep the reference while it serves: within kSpread above every scale
                        if (top > ref_b || (top && low + kSpread < ref_b)) {
                            if (ref_b) {
                                const int d = (int)ref_b - (int)top;         // exact: powers of two
                                const float f = pow2i(d / 2);
                                const float f2 = pow2i(d - d / 2);
#pragma unroll
                                for (int x = 0; x < RT; ++x)
#pragma unroll
                                    for (int n = 0; n < NO; ++n)
#pragma unroll
                                        for (int e = 0; e < 4; ++e) o[x][n][e] = o[x][n][e] * f * f2;
                            }
                            ref_b = top;
                            ref_high = max(ref_high, top);
                        }
                        const uint32_t from = ref_b > kSpread ? ref_b - kSpread : 0u;   // this pass
#pragma unroll
                        for (int h = 0; h < H; ++h)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t bb = __shfl_sync(0xffffffffu, byte, h * 16 + i * key_step + key0);
                                fv[h][i] = bb >= from && bb < below && bb != 0u
                                               ? __uint_as_float((bb + 127u + kBase - ref_b) << 23) : 0.f;
                                if (bb == kScaleNan) fv[h][i] = __int_as_float(0x7fc00000);
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
                        for (int i = 0; i < 2; ++i) {
                            const int dim = (2 * n + i) * 8 + g8;
                            float v;
                            if constexpr (kQuant) {
                                const uint8_t w = gv[j * F::kRowBytes + (((dim >> 4) ^ F::swizzle(1, j)) << 4) + (dim & 15)];
                                float f[4];
                                e4m3x4_to_f32(w, f);
                                v = f[0];      // a NaN scale came with P
                            } else {
                                v = to_f(*reinterpret_cast<const __nv_bfloat16*>(
                                    gv + j * F::kRowBytes + (((dim >> 3) ^ (j & 7)) << 4) + (dim & 7) * 2));
                            }
                            if (isfinite(v)) continue;
#pragma unroll
                            for (int r = 0; r < 2 * RT; ++r)
                                if (j0 + j <= pos[r]) o[r >> 1][n][2 * i + (r & 1)] += v;
                        }
                }
            }
        }
        cp_wait<0>();

        // ---- join the four warps
        if constexpr (kQuant) {
            const int low = (int)__reduce_min_sync(0xffffffffu, low_b) + 1;
            if (lane == 0 && (int)ref_high - low > kSpan) mark_redo(a, it);
            const float unit = ref_b ? pow2i((int)ref_b - 127 - kBase) : 0.f;
#pragma unroll
            for (int x = 0; x < RT; ++x)
#pragma unroll
                for (int n = 0; n < NO; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[x][n][e] *= unit;
        }
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r)
#pragma unroll
            for (int d = 4; d < 32; d *= 2) l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
        __syncthreads();                       // every warp has left its ring
        float* mo = reinterpret_cast<float*>(ring);                  // [warp][row][kMergeLd]
        float* mm = mo + kWarps * F::kRows * F::kMergeLd;            // [warp][row] maxima
        float* ml = mm + kWarps * F::kRows;                          // sums
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) {
            const int row = 8 * (r >> 1) + 2 * t4 + (r & 1);
            float* d = mo + (warp * F::kRows + row) * F::kMergeLd;
#pragma unroll
            for (int n = 0; n < NO; ++n) {
                d[2 * n * 8 + g8] = o[r >> 1][n][r & 1];
                d[(2 * n + 1) * 8 + g8] = o[r >> 1][n][2 + (r & 1)];
            }
            if (g8 == 0) {
                mm[warp * F::kRows + row] = m[r];
                ml[warp * F::kRows + row] = l[r];
            }
        }
        __syncthreads();
        constexpr int kLanes = kThreads / 8;                          // threads per row
#pragma unroll
        for (int r0 = 0; r0 < F::kRows; r0 += 8) {
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

template <int CD, int D, int RT>
cudaError_t launch(const PagedArgs& a, cudaStream_t st) {
    using F = Few<CD, D, RT>;
    static_assert(F::kSmem <= 227 * 1024 / F::kCtas - 1024, "stages exceed shared memory");
    auto kern = k_paged_few<CD, D, RT>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem((const void*)kern, F::kSmem, done);
    if (e != cudaSuccess) return e;
    int shift = 0;
    while ((1 << shift) < a.kv.page_size) ++shift;
    if ((e = launch_chained(kern, a.grid, kThreads, F::kSmem, st, a, shift))) return e;
    note_launch();
    return cudaSuccess;
}

// Applies fn.template operator()<CD, D, RT>() for the call's shape.
template <int CD, class Fn>
auto by_rows(const PagedArgs& a, Fn fn) {
    const int64_t rows = (int64_t)a.b.max_rows * (a.Hq / a.kv.Hkv);
    switch (a.kv.d) {
        case 64:
            return rows <= 8 ? fn.template operator()<CD, 64, 1>() : rows <= 16 ? fn.template operator()<CD, 64, 2>()
                 : rows <= 24 ? fn.template operator()<CD, 64, 3>() : fn.template operator()<CD, 64, 4>();
        case 128:
            return rows <= 8 ? fn.template operator()<CD, 128, 1>() : rows <= 16 ? fn.template operator()<CD, 128, 2>()
                 : rows <= 24 ? fn.template operator()<CD, 128, 3>() : fn.template operator()<CD, 128, 4>();
        default:
            return rows <= 8 ? fn.template operator()<CD, 256, 1>() : fn.template operator()<CD, 256, 2>();
    }
}
template <class Fn>
auto by_shape(const PagedArgs& a, Fn fn) {
    return a.kv.dtype == TAM_E4M3 ? by_rows<TAM_E4M3>(a, fn) : by_rows<TAM_BF16>(a, fn);
}

// An item's own cost (Q, the first loads, the join of the warps), in tiles.  One token over 4096:
// 14.7 us at 2, 14.4 at 4, 13.7 at 6, 13.8 at 9; 32 e4m3 sequences of up to 32K: 100.7, 101.4, 101.2,
// 103.8; five drafted tokens of 16 sequences: 37.5, 37.2, 37.7, 37.8.  Only the single token gains;
// the others do not depend on it up to 6.
constexpr int kStart = 6;
struct ShapeOf {
    template <int CD, int D, int RT>
    PagedShape operator()() const {
        using F = Few<CD, D, RT>;
        return {F::kRows, kWarps * F::kKeys, 148 * F::kCtas, kStart};
    }
};
struct Launch {
    const PagedArgs& a;
    cudaStream_t st;
    template <int CD, int D, int RT>
    cudaError_t operator()() const { return launch<CD, D, RT>(a, st); }
};

}  // namespace

bool paged_few_supported(const PagedArgs& a) {
    const int64_t rows = (int64_t)a.b.max_rows * (a.Hq / a.kv.Hkv);
    return a.dtype == TAM_BF16 && rows > 0 && rows <= (a.kv.d <= 128 ? 32 : 16);
}

PagedShape paged_few_shape(const PagedArgs& a) { return by_shape(a, ShapeOf{}); }

cudaError_t paged_few(const PagedArgs& a, cudaStream_t st) { return by_shape(a, Launch{a, st}); }

}  // namespace tam
