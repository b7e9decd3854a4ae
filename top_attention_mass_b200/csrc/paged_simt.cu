// Attention over pages for fp32 queries, on the CUDA cores.
//
//   x_j = scale*log2(e) * q.k_j  (j <= position),  m = max x_j,  p_j = 2^(x_j - m),
//   out = sum p_j v_j / sum p_j,  lse = ln 2 * m + ln sum p_j
//
// Products and sums in fp32.  A CTA of 128 threads takes one item
// (16 rows of a KV head's query heads) and streams key tiles of 32 through shared memory as
// fp32, with the running maximum and sum of every row; 8 threads share a row (4 keys each
// for the scores, d / 8 columns each for the output).  Bound: shared-memory reads, one
// 16-byte read per 4 FMAs.
#include "launch.h"
#include "paged.cuh"

namespace tam {
namespace {

constexpr int kRows = 16, kKeys = 32, kThreads = 128;

template <int D>
constexpr int smem_bytes() {
    return ((kRows + 2 * kKeys) * (D + 4) + kRows * (kKeys + 1)) * 4;
}

template <int CD, int D>
__global__ void __launch_bounds__(kThreads) k_paged_simt(const PagedArgs a, int page_shift) {
    using C = CacheVec<CD>;
    constexpr int LD = D + 4, PW = kKeys + 1;
    extern __shared__ float4 smem4[];
    float* sq = reinterpret_cast<float*>(smem4);
    float* sk = sq + kRows * LD;
    float* sv = sk + kKeys * LD;
    float* sp = sv + kKeys * LD;
    __shared__ int64_t at[kKeys];          // element offset of the key's row; -1: not there
    __shared__ int64_t sat[kKeys];
    const int tid = threadIdx.x, r = tid >> 3, l8 = tid & 7;
    const int G = a.Hq / a.kv.Hkv, Hkv = a.kv.Hkv;
    wait_for_previous();                       // the plan
    let_next_start();                          // the join may read the plan while this runs
    PagedWalk walk(a, blockIdx.x);
    PagedItem it;
    while (walk.next(it)) {
        const PagedBlock& k = it.blk;
        const int n_rows = (int)min((int64_t)kRows, (int64_t)k.n * G - k.row0);
        __syncthreads();
        for (int i = tid; i < kRows * D; i += kThreads) {
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
        float m = -INFINITY, l = 0.f, o[D / 8];
#pragma unroll
        for (int e = 0; e < D / 8; ++e) o[e] = 0.f;
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
            float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                const float4 q4 = *reinterpret_cast<const float4*>(sq + r * LD + c);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float4 k4 = *reinterpret_cast<const float4*>(sk + (u * 8 + l8) * LD + c);
                    x[u] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, x[u]))));
                }
            }
            float top = m;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = j0 + u * 8 + l8;
                x[u] = (j <= pos && at[u * 8 + l8] >= 0) ? x[u] * a.sl2 : -INFINITY;
                top = fmaxf(top, x[u]);
            }
#pragma unroll
            for (int s = 4; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
            const float ref = top == -INFINITY ? 0.f : top;      // a row that sees no key yet
            const float corr = exp2f(m - ref);
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float p = exp2f(x[u] - ref);
                sp[r * PW + u * 8 + l8] = p;
                sum += p;
            }
#pragma unroll
            for (int s = 4; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
            l = l * corr + sum;
            m = top;
            __syncwarp();                                        // a row's 8 threads are in one warp
#pragma unroll
            for (int e = 0; e < D / 8; ++e) o[e] *= corr;
#pragma unroll 2
            for (int j = 0; j < kKeys; ++j) {
                const float p = sp[r * PW + j];
                if (p == 0.f) continue;              // masked: no effect, whatever v holds
#pragma unroll
                for (int e = 0; e < D / 32; ++e) {
                    const float4 v4 = *reinterpret_cast<const float4*>(sv + j * LD + e * 32 + l8 * 4);
                    o[4 * e] = fmaf(p, v4.x, o[4 * e]);
                    o[4 * e + 1] = fmaf(p, v4.y, o[4 * e + 1]);
                    o[4 * e + 2] = fmaf(p, v4.z, o[4 * e + 2]);
                    o[4 * e + 3] = fmaf(p, v4.w, o[4 * e + 3]);
                }
            }
        }
        if (r >= n_rows) continue;
        if (it.slot >= 0) {
            float* p = part_slot(a, blockIdx.x, it.slot);
#pragma unroll
            for (int e = 0; e < D / 32; ++e)
                *reinterpret_cast<float4*>(p + (size_t)r * D + e * 32 + l8 * 4) =
                    make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            if (l8 == 0) {
                p[(size_t)kRows * D + r] = m;
                p[(size_t)kRows * (D + 1) + r] = l;
            }
            continue;
        }
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
        const int64_t tok = k.tok0 + row / G;
        const int h = it.g * G + (int)(row % G);
        float* out = (float*)a.out + (tok * a.Hq + h) * D;
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            *reinterpret_cast<float4*>(out + e * 32 + l8 * 4) = make_float4(
                o[4 * e] * inv, o[4 * e + 1] * inv, o[4 * e + 2] * inv, o[4 * e + 3] * inv);
        if (a.lse && l8 == 0)
            a.lse[(int64_t)a.Hq * k.tok0 + (int64_t)h * k.n + row / G] = lse_of(m, l);
    }
}

template <int CD, int D>
cudaError_t launch(const PagedArgs& a, cudaStream_t st) {
    auto kern = k_paged_simt<CD, D>;
    constexpr int smem = smem_bytes<D>();
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem((const void*)kern, smem, done);
    if (e != cudaSuccess) return e;
    int shift = 0;
    while ((1 << shift) < a.kv.page_size) ++shift;
    if ((e = launch_chained(kern, a.grid, kThreads, smem, st, a, shift))) return e;
    note_launch();
    return cudaSuccess;
}

template <int CD>
cudaError_t by_d(const PagedArgs& a, cudaStream_t st) {
    switch (a.kv.d) {
        case 64: return launch<CD, 64>(a, st);
        case 128: return launch<CD, 128>(a, st);
        default: return launch<CD, 256>(a, st);
    }
}

}  // namespace

PagedShape paged_simt_shape(const PagedArgs&) { return {kRows, kKeys, 148 * 2, 1}; }

cudaError_t paged_simt(const PagedArgs& a, cudaStream_t st) {
    return a.kv.dtype == TAM_F32 ? by_d<TAM_F32>(a, st) : by_d<TAM_E4M3>(a, st);
}

}  // namespace tam
