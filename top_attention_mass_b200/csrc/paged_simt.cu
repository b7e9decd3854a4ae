// Attention over pages for fp32 queries, on the CUDA cores.
//
//   x_j = scale*log2(e) * q.k_j  (j <= position),  m = max x_j,  p_j = 2^(x_j - m),
//   out = sum p_j v_j / sum p_j,  lse = ln 2 * m + ln sum p_j
//
// Products and sums in fp32.  A CTA of 128 threads takes one item (R = 4 or 16 rows of a KV
// head's query heads) and streams key tiles of 32 through shared memory as fp32, with the
// running maximum and sum of every row; 128 / R threads share a row (32 keys and d columns
// between them).  Bound: shared-memory reads, one 16-byte read per 4 FMAs, so that rows that
// are not there cost as much as the others: up to 8 rows go in blocks of 4, more in blocks of 16.
// Measured, one token each of 8 sequences of 1000 to 8192, d = 128, fp32 pages: 4 rows per KV head
// (32/8 heads) 183 us, 409 in blocks of 16; 8 rows (32/4) 171 us, 224; over e4m3 pages 131 us.  256
// tokens over 4096, 16/4 heads: 1.13 ms (7.4 TFLOP/s) over fp32 and over e4m3 pages.
#include "launch.h"
#include "paged.cuh"

namespace tam {
namespace {

constexpr int kKeys = 32, kThreads = 128;

// W floats of a thread's columns, 8 or 16 bytes at a time.
template <int W> struct vec;
template <> struct vec<2> {
    static __device__ __forceinline__ void load(float* v, const float* p) {
        const float2 x = *reinterpret_cast<const float2*>(p);
        v[0] = x.x; v[1] = x.y;
    }
    static __device__ __forceinline__ void store(float* p, const float* v, float f) {
        *reinterpret_cast<float2*>(p) = make_float2(v[0] * f, v[1] * f);
    }
};
template <> struct vec<4> {
    static __device__ __forceinline__ void load(float* v, const float* p) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    }
    static __device__ __forceinline__ void store(float* p, const float* v, float f) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
    }
};

template <int D, int R>
constexpr int smem_bytes() {
    return ((R + 2 * kKeys) * (D + 4) + R * (kKeys + 1)) * 4;
}

template <int CD, int D, int R>
__global__ void __launch_bounds__(kThreads) k_paged_simt(const PagedArgs a, int page_shift) {
    using C = CacheVec<CD>;
    constexpr int LD = D + 4, PW = kKeys + 1;
    constexpr int TPR = kThreads / R, KU = kKeys / TPR;           // threads per row, keys per thread
    constexpr int W = D / TPR < 4 ? 2 : 4, NE = D / TPR / W;      // vectors of its columns
    static_assert(W * NE * TPR == D, "columns");
    extern __shared__ float4 smem4[];
    float* sq = reinterpret_cast<float*>(smem4);
    float* sk = sq + R * LD;
    float* sv = sk + kKeys * LD;
    float* sp = sv + kKeys * LD;
    __shared__ int64_t at[kKeys];          // element offset of the key's row; -1: not there
    __shared__ int64_t sat[kKeys];
    const int tid = threadIdx.x, r = tid / TPR, lr = tid % TPR;
    const int G = a.Hq / a.kv.Hkv, Hkv = a.kv.Hkv;
    wait_for_previous();                       // the plan
    let_next_start();                          // the join may read the plan while this runs
    PagedWalk walk(a, blockIdx.x);
    PagedItem it;
    while (walk.next(it)) {
        const PagedBlock& k = it.blk;
        const int n_rows = (int)min((int64_t)R, (int64_t)k.n * G - k.row0);
        __syncthreads();
        for (int i = tid; i < R * D; i += kThreads) {
            const int rr = i / D, c = i % D;
            float x = 0.f;
            if (rr < n_rows) {
                const int64_t row = (int64_t)k.row0 + rr;
                x = ((const float*)a.q)[((k.tok0 + row / G) * a.Hq + it.g * G + row % G) * D + c];
            }
            sq[rr * LD + c] = x;
        }
        const int64_t row = (int64_t)k.row0 + r;
        const int pos = r < n_rows ? k.pos0 + (int)(row / G) : -1;
        float m = -INFINITY, l = 0.f, o[D / TPR];
#pragma unroll
        for (int e = 0; e < D / TPR; ++e) o[e] = 0.f;
        for (int t = it.t0; t < it.t1; ++t) {
            const int j0 = t * kKeys;
            __syncthreads();
            if (tid < kKeys) {
                const int j = j0 + tid;
                int64_t off = -1, soff = 0;
                if (j < k.len) {
                    const int page = page_of(a.b, a.kv, k.seq, page_shift, j, a.status, KID_PAGED_SIMT);
                    if (page >= 0) {
                        const int in = j & (a.kv.page_size - 1);
                        off = page * a.kv.page_stride + in * a.kv.row_stride + it.g * a.kv.head_stride;
                        soff = (((int64_t)page * Hkv + it.g) << page_shift) + in;
                    }
                }
                at[tid] = off;
                sat[tid] = soff;
            }
            __syncthreads();
            constexpr int VPR = D / C::N;
            for (int i = tid; i < 2 * kKeys * VPR; i += kThreads) {
                const int x = i / (kKeys * VPR), j = i / VPR % kKeys, c = i % VPR;
                float f[C::N];
#pragma unroll
                for (int e = 0; e < C::N; ++e) f[e] = 0.f;
                if (at[j] >= 0) {
                    const uint8_t* p = (const uint8_t*)(x ? a.kv.v_pages : a.kv.k_pages);
                    float s = 1.f;
                    if constexpr (CD == TAM_E4M3) s = scale_value((x ? a.kv.v_scale : a.kv.k_scale)[sat[j]]);
                    C::to_f32(*reinterpret_cast<const uint4*>(p + (at[j] + c * C::N) * C::kBytes), s, f);
                }
                float* d = (x ? sv : sk) + j * LD + c * C::N;
#pragma unroll
                for (int e = 0; e < C::N; e += 4)
                    *reinterpret_cast<float4*>(d + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
            }
            __syncthreads();
            float x[KU];
#pragma unroll
            for (int u = 0; u < KU; ++u) x[u] = 0.f;
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                const float4 q4 = *reinterpret_cast<const float4*>(sq + r * LD + c);
#pragma unroll
                for (int u = 0; u < KU; ++u) {
                    const float4 k4 = *reinterpret_cast<const float4*>(sk + (u * TPR + lr) * LD + c);
                    x[u] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, x[u]))));
                }
            }
            float top = m;
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                const int j = j0 + u * TPR + lr;
                x[u] = (j <= pos && at[u * TPR + lr] >= 0) ? x[u] * a.sl2 : -INFINITY;
                top = fmaxf(top, x[u]);
            }
#pragma unroll
            for (int s = TPR / 2; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
            const float ref = top == -INFINITY ? 0.f : top;      // a row that sees no key yet
            const float corr = exp2f(m - ref);
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                const float p = exp2f(x[u] - ref);
                sp[r * PW + u * TPR + lr] = p;
                sum += p;
            }
#pragma unroll
            for (int s = TPR / 2; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
            l = l * corr + sum;
            m = top;
            __syncwarp();                                        // a row's threads are in one warp
#pragma unroll
            for (int e = 0; e < D / TPR; ++e) o[e] *= corr;
#pragma unroll 2
            for (int j = 0; j < kKeys; ++j) {
                const float p = sp[r * PW + j];
                if (p == 0.f) continue;              // masked: no effect, whatever v holds
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    float v[W];
                    vec<W>::load(v, sv + j * LD + (e * TPR + lr) * W);
#pragma unroll
                    for (int c = 0; c < W; ++c) o[W * e + c] = fmaf(p, v[c], o[W * e + c]);
                }
            }
        }
        if (r >= n_rows) continue;
        if (it.slot >= 0) {
            float* p = part_slot(a, blockIdx.x, it.slot);
#pragma unroll
            for (int e = 0; e < NE; ++e) vec<W>::store(p + (size_t)r * D + (e * TPR + lr) * W, o + W * e, 1.f);
            if (lr == 0) {
                p[(size_t)R * D + r] = m;
                p[(size_t)R * (D + 1) + r] = l;
            }
            continue;
        }
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
        const int64_t tok = k.tok0 + row / G;
        const int h = it.g * G + (int)(row % G);
        float* out = (float*)a.out + (tok * a.Hq + h) * D;
#pragma unroll
        for (int e = 0; e < NE; ++e) vec<W>::store(out + (e * TPR + lr) * W, o + W * e, inv);
        if (a.lse && lr == 0)
            a.lse[(int64_t)a.Hq * k.tok0 + (int64_t)h * k.n + row / G] = lse_of(m, l);
    }
}

template <int CD, int D, int R>
cudaError_t launch(const PagedArgs& a, cudaStream_t st) {
    auto kern = k_paged_simt<CD, D, R>;
    constexpr int smem = smem_bytes<D, R>();
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem((const void*)kern, smem, done);
    if (e != cudaSuccess) return e;
    int shift = 0;
    while ((1 << shift) < a.kv.page_size) ++shift;
    if ((e = launch_chained(kern, a.grid, kThreads, smem, st, a, shift))) return e;
    note_launch();
    return cudaSuccess;
}

// Few rows per sequence and KV head: blocks of 4 (figures at the top).
bool few(const PagedArgs& a) {
    const int64_t rows = (int64_t)a.b.max_rows * (a.Hq / a.kv.Hkv);
    return rows > 0 && rows <= 8;
}

template <int CD>
cudaError_t by_d(const PagedArgs& a, cudaStream_t st) {
    switch (a.kv.d) {
        case 64: return few(a) ? launch<CD, 64, 4>(a, st) : launch<CD, 64, 16>(a, st);
        case 128: return few(a) ? launch<CD, 128, 4>(a, st) : launch<CD, 128, 16>(a, st);
        default: return few(a) ? launch<CD, 256, 4>(a, st) : launch<CD, 256, 16>(a, st);
    }
}

}  // namespace

PagedShape paged_simt_shape(const PagedArgs& a) {
    if (few(a)) return {4, kKeys, 148 * (a.kv.d <= 128 ? 4 : 3), 1};
    return {16, kKeys, 148 * 2, 1};
}

cudaError_t paged_simt(const PagedArgs& a, cudaStream_t st) {
    return a.kv.dtype == TAM_F32 ? by_d<TAM_F32>(a, st) : by_d<TAM_E4M3>(a, st);
}

}  // namespace tam
