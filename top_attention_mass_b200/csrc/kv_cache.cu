// The paged KV cache's own movements: new K/V rows into their pages (quantised to e4m3 on
// the way where the cache is) and rows back out of them.
//
//   write: e = the smallest exponent in [-100, 120] with max|x| <= 448 * 2^e over one token
//          and KV head, kept = rn_even_e4m3(x * 2^-e), scale byte = e + 127 (at e = 120
//          kept stops at 240: the next value times 2^120 is beyond fp32)
//   read:  x = kept * 2^e, exact in bf16 and fp32
//
// Bound: HBM, each byte once.  One CTA takes the K and V rows of a few consecutive tokens
// (all KV heads, so its reads of the packed side are one contiguous run per tensor); a
// thread moves 16 bytes of K and of V of kUnroll rows at once, and the
// lanes that hold one row find its maximum by shuffles.  The tokens' places in the cache are
// looked up once per CTA; the write's first loads of the rows are in flight meanwhile.  No
// integer division runs per vector (with two, the address arithmetic bound both at 77 us).
// Measured, 34642 tokens of 8 KV heads, d = 128, pages of 64 tokens, call after call with the status
// clear in front: bf16 rows and e4m3 pages (213 MB) write 45 us (4.7 TB/s, 0.72 of the measured copy
// rate), read 42 us (0.77; the kernel alone 34 us); fp32 rows and e4m3 pages (355 MB) write 71 us
// (0.76), read 70 us (0.77); bf16 pages, as they are (284 MB), write 50 us (0.86); fp32 pages (568 MB)
// read 96 us (0.90).  64 single tokens 5 to 6 us.
#include <algorithm>

#include "launch.h"
#include "paged.cuh"

namespace tam {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;          // rows in flight per thread, a 16-byte vector of K and of V each
constexpr int kPerSm = 16;          // CTAs per SM that a large call is cut into
constexpr int kMaxTokens = 64;      // tokens per CTA, at most

struct Place {
    int64_t row;      // page * page_stride + row in it * row_stride (elements); -1: none
    int64_t scale;    // page * Hkv * page_size + row in it
    bool mine;        // the packed row belongs to a sequence
};

// Places of the tokens t0 .. t0 + n_tok - 1, one thread each, by the whole block (barriers).
// A token's sequence is the number of s with cu_rows[s + 1] <= t: counted by all threads at
// once for the first and the last token, found by bisection between the two for the others,
// so that the chain of dependent loads stays short.
__device__ __forceinline__ void find_places(const KvRowsArgs& a, int page_shift, int64_t t0,
                                            int n_tok, int kid, Place* place) {
    int s0 = 0, s1 = 0;
    for (int s = 0; s < a.b.n_seq; s += kThreads) {
        const int i = s + threadIdx.x;
        const int64_t c = i < a.b.n_seq ? a.b.cu_rows[i + 1] : INT64_MAX;
        s0 += __syncthreads_count(c <= t0);
        s1 += __syncthreads_count(c <= t0 + n_tok - 1);
    }
    if (threadIdx.x < n_tok) {
        const int64_t t = t0 + threadIdx.x;
        Place r{-1, 0, false};
        int lo = s0, hi = max(s1, s0);
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.b.cu_rows[mid + 1] > t) hi = mid;
            else lo = mid + 1;
        }
        const int s = lo;
        if (s < a.b.n_seq) {
            const int64_t first = a.b.cu_rows[s], end = a.b.cu_rows[s + 1];
            const int64_t p = (int64_t)a.b.kv_len[s] - (end - t);
            r.mine = t >= first && t < end;
            if (r.mine && p >= ((int64_t)a.b.max_pages << page_shift)) {
                report_error(a.status, TAM_ERR_PAGE, kid, s, (int32_t)p, -1);
            } else if (r.mine && p >= 0) {
                const int page = page_of(a.b, a.kv, s, page_shift, (int)p, a.status, kid);
                if (page >= 0) {
                    const int row = (int)p & (a.kv.page_size - 1);
                    r.row = page * a.kv.page_stride + row * a.kv.row_stride;
                    r.scale = ((int64_t)page * a.kv.Hkv << page_shift) + row;
                }
            }
        }
        place[threadIdx.x] = r;
    }
    __syncthreads();
}

template <typename T, int D>
struct Lanes {
    static constexpr int V = 16 / (int)sizeof(T);              // elements per vector
    static constexpr int kVec = D / V;                          // vectors per row
    static constexpr int kRow = kVec < 32 ? kVec : 32;          // lanes per row
    static constexpr int kPer = kVec / kRow;                    // vectors per lane (1, or 2)
};

// Rows of the CTA (token * Hkv + head) stand in a run on the packed side; the token of row r is
// r / Hkv = r * ceil(2^32 / Hkv) >> 32, exact for r < 64 * Hkv and Hkv <= 4096.
__device__ __forceinline__ int token_of(uint32_t r, uint32_t inv) {
    return (int)(inv ? __umulhi(r, inv) : r);      // inv = 0: one head
}

template <int CD, typename T, int D>
__global__ void __launch_bounds__(kThreads) k_kv_write(const KvRowsArgs a, int page_shift, int tpb,
                                                       uint32_t inv_heads) {
    using L = Lanes<T, D>;
    constexpr int CB = CacheVec<CD>::kBytes;
    __shared__ Place place[kMaxTokens];
    const int64_t t0 = (int64_t)blockIdx.x * tpb;
    const int n_tok = (int)min((int64_t)tpb, a.T - t0);
    const int Hkv = a.kv.Hkv;
    const int total = n_tok * Hkv * L::kRow;
    const int lane = threadIdx.x % L::kRow;
    const T* src[2] = {(const T*)a.k + t0 * Hkv * D + lane * L::V,
                       (const T*)a.v + t0 * Hkv * D + lane * L::V};
    uint8_t* dst[2] = {(uint8_t*)a.kv.k_pages + lane * L::V * CB,
                       (uint8_t*)a.kv.v_pages + lane * L::V * CB};
    uint8_t* scl[2] = {a.kv.k_scale, a.kv.v_scale};
    bool placed = false;
    for (int i0 = 0; i0 < total; i0 += kThreads * kUnroll) {
        uint4 w[kUnroll][2][L::kPer];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * kThreads + threadIdx.x;
            const int64_t at = (int64_t)(i / L::kRow) * D;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int z = 0; z < L::kPer; ++z)
                    w[u][x][z] = i < total ? __ldg(reinterpret_cast<const uint4*>(
                                                 src[x] + at + z * L::kRow * L::V))
                                           : make_uint4(0, 0, 0, 0);
        }
        if (!placed) {                       // the same for every thread of the block
            find_places(a, page_shift, t0, n_tok, KID_KV_WRITE, place);
            placed = true;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * kThreads + threadIdx.x;
            const bool have = i < total;
            const int r = have ? i / L::kRow : 0;
            const int tok = token_of(r, inv_heads), g = r - tok * Hkv;
            const int64_t row = place[tok].row;
            const bool keep = have && row >= 0;
            const int64_t at = (row + g * a.kv.head_stride) * CB;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint8_t* out = dst[x] + at;
                if constexpr (CD != TAM_E4M3) {
                    if (keep)
#pragma unroll
                        for (int z = 0; z < L::kPer; ++z)
                            *reinterpret_cast<uint4*>(out + z * L::kRow * 16) = w[u][x][z];
                } else {
                    float f[L::kPer][L::V];
                    uint32_t top = 0;        // |x| as bits: ordered, infinity and NaN on top
#pragma unroll
                    for (int z = 0; z < L::kPer; ++z) {
                        CacheVec<sizeof(T) == 2 ? TAM_BF16 : TAM_F32>::to_f32(w[u][x][z], 1.f, f[z]);
#pragma unroll
                        for (int e = 0; e < L::V; ++e)
                            top = max(top, __float_as_uint(f[z][e]) & 0x7fffffffu);
                    }
#pragma unroll
                    for (int o = L::kRow / 2; o > 0; o >>= 1)
                        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    // top = 1.f * 2^(E - 127); 448 = 1.75 * 2^8
                    const int E = (int)(top >> 23);
                    int e = E - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
                    e = min(max(e, kScaleExpMin), kScaleExpMax);
                    const bool finite = top < 0x7f800000u;
                    const float inv = __int_as_float((127 - e) << 23);   // 2^-e, a normal number
                    if (!keep) continue;
#pragma unroll
                    for (int z = 0; z < L::kPer; ++z) {
#pragma unroll
                        for (int c = 0; c < L::V; ++c) f[z][c] *= inv;
                        // 256 * 2^120 is no fp32 number: the last value below it instead
                        if (e == kScaleExpMax)
#pragma unroll
                            for (int c = 0; c < L::V; ++c)
                                f[z][c] = fminf(fmaxf(f[z][c], -240.f), 240.f);
                        uint32_t y[L::V / 4];
#pragma unroll
                        for (int c = 0; c < L::V / 4; ++c) {
                            const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                                make_float2(f[z][4 * c], f[z][4 * c + 1]), __NV_SATFINITE,
                                __NV_E4M3);
                            const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                                make_float2(f[z][4 * c + 2], f[z][4 * c + 3]), __NV_SATFINITE,
                                __NV_E4M3);
                            y[c] = finite ? (lo | (hi << 16)) : 0u;
                        }
                        if constexpr (L::V == 8)
                            *reinterpret_cast<uint2*>(out + z * L::kRow * L::V) = make_uint2(y[0], y[1]);
                        else
                            *reinterpret_cast<uint32_t*>(out + z * L::kRow * L::V) = y[0];
                    }
                    if (lane == 0)
                        scl[x][place[tok].scale + ((int64_t)g << page_shift)] =
                            (uint8_t)(finite ? (uint32_t)(e + kScaleBias) : kScaleNan);
                }
            }
        }
    }
}

template <int CD, typename T, int D>
__global__ void __launch_bounds__(kThreads) k_kv_read(const KvRowsArgs a, int page_shift, int tpb,
                                                      uint32_t inv_heads) {
    constexpr int V = 16 / (int)sizeof(T), kRow = D / V;        // vectors per row
    constexpr int CB = CacheVec<CD>::kBytes;
    __shared__ Place place[kMaxTokens];
    const int64_t t0 = (int64_t)blockIdx.x * tpb;
    const int n_tok = (int)min((int64_t)tpb, a.T - t0);
    const int Hkv = a.kv.Hkv;
    const int total = n_tok * Hkv * kRow;
    const int lane = threadIdx.x % kRow;
    const uint8_t* src[2] = {(const uint8_t*)a.kv.k_pages + lane * V * CB,
                             (const uint8_t*)a.kv.v_pages + lane * V * CB};
    const uint8_t* scl[2] = {a.kv.k_scale, a.kv.v_scale};
    T* dst[2] = {(T*)a.k + t0 * Hkv * D + lane * V, (T*)a.v + t0 * Hkv * D + lane * V};
    find_places(a, page_shift, t0, n_tok, KID_KV_READ, place);
    for (int i0 = 0; i0 < total; i0 += kThreads * kUnroll) {
        uint4 w[kUnroll][2];
        uint32_t sc[kUnroll][2];
        bool mine[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * kThreads + threadIdx.x;
            mine[u] = i < total;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                w[u][x] = make_uint4(0, 0, 0, 0);
                sc[u][x] = kScaleBias;
            }
            if (i < total) {
                const int r = i / kRow;
                const int tok = token_of(r, inv_heads), g = r - tok * Hkv;
                const Place pl = place[tok];
                mine[u] = pl.mine;
                if (pl.row >= 0) {
                    const int64_t at = (pl.row + g * a.kv.head_stride) * CB;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint8_t* p = src[x] + at;
                        if constexpr (CD != TAM_E4M3) {
                            w[u][x] = __ldg(reinterpret_cast<const uint4*>(p));
                        } else {
                            if constexpr (V == 8) {
                                const uint2 y = __ldg(reinterpret_cast<const uint2*>(p));
                                w[u][x].x = y.x;
                                w[u][x].y = y.y;
                            } else {
                                w[u][x].x = __ldg(reinterpret_cast<const uint32_t*>(p));
                            }
                            sc[u][x] = __ldg(scl[x] + pl.scale + ((int64_t)g << page_shift));
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (!mine[u]) continue;
            const int64_t at = (int64_t)((i0 + u * kThreads + threadIdx.x) / kRow) * D;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint4 y = w[u][x];
                if constexpr (CD == TAM_E4M3) {
                    const float s = scale_value(sc[u][x]);
                    uint32_t o[4];
#pragma unroll
                    for (int c = 0; c < V / 4; ++c) {
                        float f[4];
                        e4m3x4_to_f32(c ? w[u][x].y : w[u][x].x, f);
                        if constexpr (V == 8) {
                            const __nv_bfloat162 p0 = __floats2bfloat162_rn(f[0] * s, f[1] * s);
                            const __nv_bfloat162 p1 = __floats2bfloat162_rn(f[2] * s, f[3] * s);
                            o[2 * c] = *reinterpret_cast<const uint32_t*>(&p0);
                            o[2 * c + 1] = *reinterpret_cast<const uint32_t*>(&p1);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[e] = __float_as_uint(f[e] * s);
                        }
                    }
                    y = make_uint4(o[0], o[1], o[2], o[3]);
                }
                *reinterpret_cast<uint4*>(dst[x] + at) = y;
            }
        }
    }
}

// Tokens per CTA.  The look-up of the places is a chain of loads that costs about as much as
// two rounds of loads, so a CTA takes as many tokens as leave kPerSm CTAs per SM (8 are
// resident: 16 measured 40.7 us for the read below, 8 45.4 us, 4 43.2 us), up to kMaxTokens; and
// never less than one row per thread.
int tokens_per_cta(int64_t T, int lanes_per_token) {
    const int64_t n = std::max<int64_t>((T + 148 * kPerSm - 1) / (148 * kPerSm),
                                        kThreads / lanes_per_token);
    return (int)std::min<int64_t>(std::max<int64_t>(n, 1), kMaxTokens);
}

int shift_of(int page_size) {
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

template <bool kWrite, int CD, typename T, int D>
cudaError_t launch(const KvRowsArgs& a, cudaStream_t st) {
    const int lanes = kWrite ? Lanes<T, D>::kRow : D / (16 / (int)sizeof(T));
    const int tpb = tokens_per_cta(a.T, a.kv.Hkv * lanes);
    const uint32_t inv = a.kv.Hkv == 1 ? 0 : (uint32_t)(((uint64_t(1) << 32) + a.kv.Hkv - 1) / a.kv.Hkv);
    const unsigned grid = (unsigned)((a.T + tpb - 1) / tpb);
    const int shift = shift_of(a.kv.page_size);
    if constexpr (kWrite) k_kv_write<CD, T, D><<<grid, kThreads, 0, st>>>(a, shift, tpb, inv);
    else k_kv_read<CD, T, D><<<grid, kThreads, 0, st>>>(a, shift, tpb, inv);
    note_launch();
    return cudaGetLastError();
}

template <bool kWrite, int CD, typename T>
cudaError_t by_d(const KvRowsArgs& a, cudaStream_t st) {
    switch (a.kv.d) {
        case 64: return launch<kWrite, CD, T, 64>(a, st);
        case 128: return launch<kWrite, CD, T, 128>(a, st);
        default: return launch<kWrite, CD, T, 256>(a, st);
    }
}

template <bool kWrite>
cudaError_t by_type(const KvRowsArgs& a, cudaStream_t st) {
    switch (a.kv.dtype) {
        case TAM_BF16: return by_d<kWrite, TAM_BF16, __nv_bfloat16>(a, st);
        case TAM_F32: return by_d<kWrite, TAM_F32, float>(a, st);
        default:
            return a.dtype == TAM_F32 ? by_d<kWrite, TAM_E4M3, float>(a, st)
                                      : by_d<kWrite, TAM_E4M3, __nv_bfloat16>(a, st);
    }
}

}  // namespace

cudaError_t kv_write(const KvRowsArgs& a, cudaStream_t st) { return by_type<true>(a, st); }
cudaError_t kv_read(const KvRowsArgs& a, cudaStream_t st) { return by_type<false>(a, st); }

}  // namespace tam
