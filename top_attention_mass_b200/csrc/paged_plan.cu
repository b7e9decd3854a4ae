// Plan and join of the attention over pages (tam_paged_gqa_attention).
//
// The lengths live on the device, so the work is laid out there: k_paged_plan (one CTA)
// clears the status block, lists the row blocks of every sequence (last block first: its
// rows see the most keys) with the key tiles each one sees, and decides how the items
// (row block, KV head) go to the CTAs of the main kernel: whole where there are kWholeItems
// or more per CTA, else split evenly by tiles (PagedWalk).  k_paged_join adds up the partial
// results of split items:
//   M = max_c m_c,  out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c
// over the CTAs c of the item in order, so the result does not depend on their timing.
//
// 16-bit products over e4m3 pages hold a key tile's scales within some powers of two of one
// another.  Items where they lie further apart (the main kernels mark them: mark_redo) are
// computed here instead, in fp32 on the CUDA cores (redo_items).
#include <type_traits>

#include "launch.h"
#include "paged.cuh"

namespace tam {
namespace {

constexpr int kPlanThreads = 1024;          // 256 for small batches
constexpr int kWholeItems = 8;

__global__ void __launch_bounds__(kPlanThreads) k_paged_plan(const PagedArgs a) {
    extern __shared__ int4 seqs[];              // [n_seq] (first row, rows, keys, first position)
    int* blk0 = reinterpret_cast<int*>(seqs + a.b.n_seq);   // [n_seq + 1] first block
    __shared__ int warp_tot[33];
    __shared__ long long unit_tot[33];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
    const int G = a.Hq / a.kv.Hkv, n_seq = a.b.n_seq;
    const int64_t cap = (int64_t)a.b.max_pages * a.kv.page_size;
    let_next_start();
    if (tid < (int)(kStatusBytes / 4)) a.status[tid] = 0;
    __syncthreads();
    int base = 0;
    bool back = false;                          // some cu_rows decrease
    for (int s0 = 0; s0 < n_seq; s0 += nt) {
        const int s = s0 + tid;
        int nb = 0;
        if (s < n_seq) {
            const int64_t kv_len = a.b.kv_len[s];
            const int64_t c0 = min(max((int64_t)a.b.cu_rows[s], (int64_t)0), a.T);
            const int64_t c1 = min(max((int64_t)a.b.cu_rows[s + 1], c0), a.T);
            const int n = (int)(c1 - c0);
            back |= a.b.cu_rows[s + 1] < a.b.cu_rows[s];
            nb = (int)(((uint32_t)n * G + a.rb - 1) / (uint32_t)a.rb);
            seqs[s] = make_int4((int)c0, n, (int)min(max(kv_len, (int64_t)0), cap),
                                (int)max(kv_len - n, -(int64_t)(1 << 30)));
            if (n > 0 && kv_len > cap)
                report_error(a.status, TAM_ERR_PAGE, KID_PAGED_PLAN, s, (int32_t)kv_len, -1);
        }
        int tot;
        const int ex = block_exclusive_scan(nb, warp_tot, &tot);
        if (s < n_seq) blk0[s] = base + ex;
        base += tot;
    }
    // sequences that overlap could ask for more blocks than there is room for, or than an int
    // counts: nothing is done.  Those that do not have at most max_blocks.
    if (__syncthreads_or(back)) {
        if (tid == 0) report_error(a.status, TAM_ERR_INVALID_ARG, KID_PAGED_PLAN);
        base = 0;
    }
    if (tid == 0) blk0[n_seq] = base;
    __syncthreads();
    const int n_blocks = base;
    long long units = 0;
    for (int b0 = 0; b0 < n_blocks; b0 += nt) {
        const int b = b0 + tid;
        PagedBlock k{};
        if (b < n_blocks) {
            int lo = 0, hi = n_seq - 1;         // the last s with blk0[s] <= b
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (blk0[mid] <= b) lo = mid;
                else hi = mid - 1;
            }
            const int s = lo;
            const int4 q = seqs[s];
            const uint32_t rows = (uint32_t)q.y * G;             // below 2^31, as all sums here
            const int nb = (int)((rows + a.rb - 1) / (uint32_t)a.rb);
            const uint32_t r0 = (uint32_t)max(nb - 1 - (b - blk0[s]), 0) * a.rb;
            const uint32_t last = min(r0 + a.rb, rows) - 1;
            const int seen = (int)min(max((int64_t)q.w + last / (uint32_t)G + 1, (int64_t)0), (int64_t)q.z);
            k.seq = s;
            k.row0 = (int)r0;
            k.tok0 = q.x;
            k.n = q.y;
            k.len = q.z;
            k.pos0 = q.w;
            k.nt = max(1, (int)((uint32_t)(seen + a.kt - 1) / (uint32_t)a.kt));
        }
        // exclusive 64-bit scan of the units
        long long x = b < n_blocks ? a.start + k.nt : 0, incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) unit_tot[warp] = incl;
        __syncthreads();
        if (warp == 0) {
            const long long t = lane < nt / 32 ? unit_tot[lane] : 0;
            long long ti = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, ti, o);
                if (lane >= o) ti += y;
            }
            unit_tot[lane] = ti - t;
            if (lane == 31) unit_tot[32] = ti;
        }
        __syncthreads();
        if (b < n_blocks) {
            k.unit0 = units + unit_tot[warp] + incl - x;
            a.blocks[b] = k;
        }
        units += unit_tot[32];
        __syncthreads();
    }
    if (a.redo) {
        if (tid == 0) a.redo[0] = 0;
        for (int i = tid; i < n_blocks * a.kv.Hkv; i += nt) a.redo[kRedoMarks + i] = 0;
    }
    if (tid == 0) {
        a.plan->n_blocks = n_blocks;
        a.plan->whole = (int64_t)n_blocks * a.kv.Hkv >= (int64_t)kWholeItems * a.grid;
        const int64_t all = units * a.kv.Hkv;
        const int64_t each = div_small(all, a.grid);
        a.plan->each = each;
        a.plan->rest = (int)(all - each * a.grid);
    }
}

constexpr int kJoinThreads = 256, kJoinRows = 32;     // 4 rows per warp

// The marked items, kRedoRows rows at a time and CTA by CTA: the formula as it stands, over the keys
// each row sees, with K and V as their exact fp32 values.  The warps take 32 keys in turn; a lane
// has a key of its own for the scores and columns of its own for the sums, and the warps' sums are
// joined through shared memory, in order.  (Every item marked, 32 single tokens over 1000 to 32768,
// 16/4 heads, d = 128: 1.5 ms, 104 us with none; 1024 tokens over 8192, 32/8 heads: 9.2 ms, 15 TFLOP/s
// of FMAs and conversions, 0.21 ms with none.)
constexpr int kRedoRows = 4, kRedoWarps = kJoinThreads / 32;

template <int D>
struct RedoSmem {
    float o[kRedoWarps][D], m[kRedoWarps], l[kRedoWarps];
};

template <int D>
__device__ __noinline__ void redo_items(const PagedArgs a, int count, RedoSmem<D>& sm) {
    constexpr int R = kRedoRows, C = D / 32, B = D == 256 ? 4 : 8;   // columns per lane, V rows in flight
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = a.Hq / a.kv.Hkv, Hkv = a.kv.Hkv;
    const int page_shift = __ffs(a.kv.page_size) - 1;
    const uint8_t* const kp = (const uint8_t*)a.kv.k_pages;
    const uint8_t* const vp = (const uint8_t*)a.kv.v_pages;
    const __nv_bfloat16* const q = (const __nv_bfloat16*)a.q;
    const int64_t n_items = (int64_t)a.plan->n_blocks * Hkv;
    const int per = (a.rb + R - 1) / R;
    const int64_t units = min((int64_t)count, n_items) * per;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int item = a.redo[kRedoMarks + a.redo_items + u / per];
        if (item < 0 || item >= n_items) continue;           // never; nothing wild is read
        const PagedBlock k = a.blocks[item / Hkv];
        const int g = item % Hkv, r0 = (int)(u % per) * R;
        const int n_rows = (int)min((int64_t)min(R, a.rb - r0), (int64_t)k.n * G - k.row0 - r0);
        if (n_rows <= 0) continue;
        int64_t at_q[R];                                     // of a row's q and out
        int last[R], end = 0;                                // the last key it sees; all of them
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = k.row0 + r0 + min(r, n_rows - 1);
            at_q[r] = ((int64_t)(k.tok0 + row / G) * a.Hq + g * G + row % G) * D;
            last[r] = min(k.pos0 + row / G, k.len - 1);
            end = max(end, last[r] + 1);
        }
        float m[R], l[R], o[R][C];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) o[r][c] = 0.f;
        }
        for (int j0 = warp * 32; j0 < end; j0 += kRedoWarps * 32) {
            const int j = j0 + lane;
            int id = -1;
            int64_t at = 0;
            float vs = 0.f, x[R];
#pragma unroll
            for (int r = 0; r < R; ++r) x[r] = 0.f;
            if (j < end) id = a.b.page_table[(int64_t)k.seq * a.b.max_pages + (j >> page_shift)];
            if ((uint32_t)id >= (uint32_t)a.kv.n_pages) id = -1;             // reported already
            if (id >= 0) {
                const int in = j & (a.kv.page_size - 1);
                const int64_t sat = (((int64_t)id * Hkv + g) << page_shift) + in;
                at = id * a.kv.page_stride + in * a.kv.row_stride + g * a.kv.head_stride;
                const float ks = scale_value(a.kv.k_scale[sat]);
                vs = scale_value(a.kv.v_scale[sat]);
#pragma unroll 2
                for (int c = 0; c < D; c += 16) {
                    float f[16];
                    CacheVec<TAM_E4M3>::to_f32(*reinterpret_cast<const uint4*>(kp + at + c), ks, f);
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float y[8];
                            CacheVec<TAM_BF16>::to_f32(
                                __ldg(reinterpret_cast<const uint4*>(q + at_q[r] + c + 8 * h)), 1.f, y);
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[r] = fmaf(y[e], f[8 * h + e], x[r]);
                        }
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float s = id >= 0 && j <= last[r] ? x[r] * a.sl2 : -INFINITY;
                const float top = fmaxf(m[r], warp_max(s)), ref = top == -INFINITY ? 0.f : top;
                const float corr = exp2f(m[r] - ref);
                x[r] = exp2f(s - ref);
                l[r] = l[r] * corr + warp_sum(x[r]);
                m[r] = top;
#pragma unroll
                for (int c = 0; c < C; ++c) o[r][c] *= corr;
            }
            const int n = min(32, end - j0);
            for (int i0 = 0; i0 < n; i0 += B) {
                float f[B][C];
#pragma unroll
                for (int i = 0; i < B; ++i) {                // (zeros where there is no page)
                    const bool there = __shfl_sync(0xffffffffu, id, i0 + i) >= 0;
                    const uint8_t* p = vp + __shfl_sync(0xffffffffu, at, i0 + i) + lane * C;
                    const float s = __shfl_sync(0xffffffffu, vs, i0 + i);
                    uint32_t w[2] = {0, 0};
                    if (there) {
                        if constexpr (C == 2) {
                            w[0] = *reinterpret_cast<const uint16_t*>(p);
                        } else if constexpr (C == 4) {
                            w[0] = *reinterpret_cast<const uint32_t*>(p);
                        } else {
                            const uint2 y = *reinterpret_cast<const uint2*>(p);
                            w[0] = y.x; w[1] = y.y;
                        }
                    }
#pragma unroll
                    for (int z = 0; z < (C + 3) / 4; ++z) {
                        float y[4];
                        e4m3x4_to_f32(w[z], y);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (4 * z + e < C) f[i][4 * z + e] = y[e] * s;
                    }
                }
#pragma unroll
                for (int i = 0; i < B; ++i)
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float p = __shfl_sync(0xffffffffu, x[r], i0 + i);
                        if (j0 + i0 + i > last[r]) continue; // no effect, whatever V holds
#pragma unroll
                        for (int c = 0; c < C; ++c) o[r][c] = fmaf(p, f[i][c], o[r][c]);
                    }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r >= n_rows) break;                          // the same in the whole CTA
            __syncthreads();
#pragma unroll
            for (int c = 0; c < C; ++c) sm.o[warp][lane * C + c] = o[r][c];
            if (lane == 0) {
                sm.m[warp] = m[r];
                sm.l[warp] = l[r];
            }
            __syncthreads();
            float M = -INFINITY, sum = 0.f, y = 0.f;
            for (int w = 0; w < kRedoWarps; ++w) M = fmaxf(M, sm.m[w]);
            const float ref = M == -INFINITY ? 0.f : M;
            const int c = threadIdx.x;
            for (int w = 0; w < kRedoWarps; ++w) {
                const float f = exp2f(sm.m[w] - ref);
                sum += f * sm.l[w];
                if (c < D) y += f * sm.o[w][c];
            }
            const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
            if (c < D) ((__nv_bfloat16*)a.out)[at_q[r] + c] = __float2bfloat16_rn(y * inv);
            const int row = k.row0 + r0 + r;
            if (a.lse && c == 0)
                a.lse[(int64_t)a.Hq * k.tok0 + (int64_t)(g * G + row % G) * k.n + row / G] = lse_of(M, sum);
        }
    }
}

// One CTA per boundary between two runs and kJoinRows rows: the item that crosses it, if it
// is the first boundary the item crosses.  One warp per row; lanes own interleaved groups of
// columns.
template <typename T, int D, bool kRedo>
__global__ void __launch_bounds__(kJoinThreads) k_paged_join(const PagedArgs a) {
    // The main kernel lets this one start once the plan is there: what to join is found out while
    // it runs.  Every CTA waits for its end, with or without work: what follows in the stream
    // follows this kernel.  Until then the plan is read from L2, where its kernel has left it:
    // the main kernel has waited for that, this one not yet.
    const PagedPlan plan = ld_l2(a.plan);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = a.Hq / a.kv.Hkv, Hkv = a.kv.Hkv, rb = a.rb;
    const int chunks = (rb + kJoinRows - 1) / kJoinRows;
    const int edge = blockIdx.x / chunks + 1;                // between the runs edge - 1 and edge
    PagedBlock k{};
    int b = 0, g = 0, c0 = 0, c1 = 0;
    int64_t start = 0;
    bool mine = false;
    const int64_t x = run_start(plan, edge);
    if (!plan.whole && plan.n_blocks > 0 && x < run_start(plan, edge + 1)) {
        b = block_of(a.blocks, plan.n_blocks, Hkv, x);
        k = ld_l2(a.blocks + b);
        const int units = a.start + k.nt;
        g = (int)div_small(x - k.unit0 * Hkv, units);
        start = k.unit0 * Hkv + (int64_t)g * units;
        c0 = run_of(plan, start + a.start);                  // of its tiles
        c1 = run_of(plan, start + units - 1);
        mine = c0 == edge - 1 && c1 >= edge;   // else they start here, or crossed an edge before
    }
    wait_for_previous();
    // loaded while the parts are added up
    const int n_redo = kRedo ? a.redo[0] : 0;
    const bool marked = kRedo && mine && a.redo[kRedoMarks + b * Hkv + g] != 0;
    const int r_first = blockIdx.x % chunks * kJoinRows;
    const int r_end = mine ? (int)min((int64_t)min(rb, r_first + kJoinRows), (int64_t)k.n * G - k.row0) : 0;
    for (int r = r_first + warp; r < r_end; r += kJoinThreads / 32) {
        const int row = k.row0 + r;
        // slot of CTA c: its first, except where the item starts inside the run of c0
        const int slot0 = run_start(plan, c0) >= start ? 0 : 1;
        const size_t part = paged_part_floats(rb, D);
        const float* p0 = a.part + (size_t)c0 * 2 * part;
        auto slot_of = [&](int c) { return p0 + ((size_t)(c - c0) * 2 + (c == c0 ? slot0 : 0)) * part; };
        float acc[D / 32], sum = 0.f, M = -INFINITY;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
        // B parts in flight, the first of them while the maximum is found (one token over 4096, 37
        // parts per row: 14.7 us for the three launches, 15.8 with 8 in flight behind the maximum)
        auto add_parts = [&](auto b_tag) {
            constexpr int B = decltype(b_tag)::value;
            float2 o[B][D / 64];
            auto load = [&](int c) {
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    const float* p = slot_of(min(c + i, c1)) + (size_t)r * D + lane * 2;
#pragma unroll
                    for (int e = 0; e < D / 64; ++e) o[i][e] = *reinterpret_cast<const float2*>(p + e * 64);
                }
            };
            float m = -INFINITY, l = 0.f;                    // of the part c0 + lane
            auto load_sums = [&](int c) {
                m = -INFINITY;
                if (c > c1) return;
                const float* p = slot_of(c) + (size_t)rb * D + r;
                m = p[0];
                l = p[rb];
            };
            load_sums(c0 + lane);
            load(c0);
            M = m;
            for (int c = c0 + 32 + lane; c <= c1; c += 32) M = fmaxf(M, slot_of(c)[(size_t)rb * D + r]);
            M = warp_max(M);
            const float base = M == -INFINITY ? 0.f : M;
            for (int cc = c0; cc <= c1; cc += 32) {          // 32 weights at a time, one per lane
                if (cc != c0) load_sums(cc + lane);
                const float f = exp2f(m - base);
                sum += f * l;
                const int n = min(32, c1 - cc + 1);
                for (int i0 = 0; i0 < n; i0 += B) {
                    if (cc != c0 || i0) load(cc + i0);
#pragma unroll
                    for (int i = 0; i < B; ++i) {
                        const float fi = __shfl_sync(0xffffffffu, f, i0 + i);
                        if (i0 + i >= n) continue;
#pragma unroll
                        for (int e = 0; e < D / 64; ++e) {
                            acc[2 * e] += fi * o[i][e].x;
                            acc[2 * e + 1] += fi * o[i][e].y;
                        }
                    }
                }
            }
        };
        // most items of long chunks are in two parts, of single tokens in many
        if (c1 - c0 < 2) add_parts(std::integral_constant<int, 2>{});
        else add_parts(std::integral_constant<int, D == 256 ? 8 : 16>{});
        sum = warp_sum(sum);
        const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        if (marked) continue;                                // written below
        const int64_t tok = k.tok0 + row / G;
        const int h = g * G + row % G;
        T* o = (T*)a.out + (tok * a.Hq + h) * D;
#pragma unroll
        for (int e = 0; e < D / 64; ++e) {
            const float x = acc[2 * e] * inv, y = acc[2 * e + 1] * inv;
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<__nv_bfloat162*>(o + e * 64 + lane * 2) = __floats2bfloat162_rn(x, y);
            else
                *reinterpret_cast<float2*>(o + e * 64 + lane * 2) = make_float2(x, y);
        }
        if (a.lse && lane == 0)
            a.lse[(int64_t)a.Hq * k.tok0 + (int64_t)h * k.n + row / G] = lse_of(M, sum);
    }
    if constexpr (kRedo) {
        __shared__ RedoSmem<D> sm;
        if (n_redo) redo_items<D>(a, n_redo, sm);
    }
}

template <typename T>
cudaError_t join(const PagedArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.grid - 1) * ((a.rb + kJoinRows - 1) / kJoinRows));
    auto kern = a.kv.d == 64 ? k_paged_join<T, 64, false> : a.kv.d == 128 ? k_paged_join<T, 128, false> : k_paged_join<T, 256, false>;
    if constexpr (sizeof(T) == 2)
        if (a.redo)
            kern = a.kv.d == 64 ? k_paged_join<T, 64, true> : a.kv.d == 128 ? k_paged_join<T, 128, true> : k_paged_join<T, 256, true>;
    const cudaError_t e = launch_chained(kern, grid, kJoinThreads, 0, st, a);
    if (e != cudaSuccess) return e;
    note_launch();
    return cudaSuccess;
}

}  // namespace

cudaError_t paged_plan(const PagedArgs& a, cudaStream_t st) {
    const int smem = a.b.n_seq * 20 + 4;
    if (smem > 40 * 1024) {
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = allow_smem((const void*)k_paged_plan, kMaxPlanSeqs * 20 + 4, done);
        if (e != cudaSuccess) return e;
    }
    const int threads = a.b.n_seq <= 256 && a.max_blocks <= 256 ? 256 : kPlanThreads;
    k_paged_plan<<<1, threads, smem, st>>>(a);
    note_launch();
    return cudaGetLastError();
}

cudaError_t paged_join(const PagedArgs& a, cudaStream_t st) {
    return a.dtype == TAM_F32 ? join<float>(a, st) : join<__nv_bfloat16>(a, st);
}

}  // namespace tam
