// Attention over pages for chunks of new tokens, on the tensor cores (tcgen05).
//
//   x_j = scale*log2(e) * q.k_j,  out = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m)
//
// Bound: tensor cores for long chunks (every K/V tile serves 128 or 256 rows), HBM for short
// ones.  The rows of an item are (token, query head of the KV group), packed densely for any
// group size.  K and V come page by page through TMA into one ring of tiles; S = Q K^T and
// O += P V accumulate in TMEM.  P never leaves TMEM: the softmax warps read S into registers and
// store P over it as 16-bit pairs, where the P V product takes it as its A operand.
//
// One softmax warpgroup alone leaves the tensor cores idle while it computes, so two work in
// turns ("channels", each with its own S/P and O columns):
//   kRows    256 rows: channel = half of the rows, both use every tile;
//   kKeys    128 rows: channel = every other key tile, joined at the end (few rows per
//            sequence: the second half of the rows would be empty);
//   kSingle  128 rows at d = 256, whose O takes the columns of two: one warpgroup, two S
//            buffers, tiles of 64 keys.
// Issue order (kRows): PV_A(t) S_A(t+1) PV_B(t) S_B(t+1): while one channel's softmax runs, the
// other channel's products do.  tcgen05.mma of one thread run in order, so S(t+1) may take the
// columns that P(t) of its channel held.
//
// e4m3: raw tiles land in a ring of their own; four warps widen them to fp16 into the tile ring.
// A row's scale enters as 2^(e - E + 7), E the largest exponent of the tile, exact down to
// 2^-22 of the tile's largest row.  An item with a K row below that (the larger one may stand where
// other rows do not see it) is computed again by the join; E itself goes into the scores
// (K) or into P's exponent (V): O is kept in units of a running exponent R that follows E when
// E > R or E < R - kSpread, and P, kept times 2^kBase, is off by 2^-25 of the largest at most
// (E = R - kSpread).  An item whose V scales span more than 2^kSpan is computed again by the join
// (small probabilities of the largest rows would lose their bits; further apart, O would overflow,
// or vanish in rows that do not see the largest); rows of zeros do not count.  Q is scaled per row by a power of two into fp16's range.
//
// What bounds it: a channel's turn is its softmax (some 2000 cycles: 128 exponentials per thread
// at 8 cycles per warp, read and written through TMEM), the rest of its P V and its next S; the
// tensor cores work 60 % of it.  Measured (device time of the three launches, behind a read of 320 MB),
// 4096 new tokens over 16384, d = 128, 32/8 heads: bf16 850 us (1132 TFLOP/s, 0.70 of the measured
// cuBLAS burst), e4m3 1088 us (885); d = 256, 16/8: 1130 us (852).  Called without a pause they draw
// the GPU's full power and the clock falls: 910, 1075, 1180 us.  512 tokens over 16384, d = 256, 16/8:
// bf16 197 us, e4m3 266 us.  24 sequences of 5 to 681 new tokens over 809 to 7049: bf16 655 us, e4m3
// 768 us.
// Tried and slower: tiles of 64 keys with two S buffers per channel (880 TFLOP/s: an MMA of N = 64
// takes as long as one of N = 128), an issuer warp per channel (1058: the channels fall into
// step), part of the exponentials on the FMA pipe (one pair in four 1081, in eight 1103, none 1102).
//
// V where it must not count: 0 times NaN is NaN, so in the tiles that some row does not see
// whole ("cut"), values that are not finite are taken out of V before the product and added to
// the rows that do see them at the end; rows behind the sequence are cleared.
#include <type_traits>

#include "launch.h"
#include "paged.cuh"
#include "tc_ptx.cuh"
#include "tma_host.h"

namespace tam {
namespace {

enum Mode { kRows = 0, kKeys = 1, kSingle = 2 };

// The row maximum is raised lazily: P goes up to 2^kLazy (e4m3: kept times 2^kBase, 2^15 in all).
constexpr float kLazy = 7.f;
constexpr int kBase = 8, kSpread = 8;
// The scales of a tile that fp16 holds exactly: an e4m3 value times 2^(e - E + 7) is a multiple of
// 2^-24 (fp16's smallest) for e >= E - 22.
constexpr int kExact = 22;

template <int CD, int D, int MODE>
struct Tc {
    static constexpr bool kQuant = CD == TAM_E4M3;
    static constexpr int kGroups = MODE == kSingle ? 1 : 2;       // softmax warpgroups
    static constexpr int kQTiles = MODE == kRows ? 2 : 1;
    static constexpr int kRb = 128 * kQTiles;
    static constexpr int KT = D == 256 ? 64 : 128;                // keys per tile
    static constexpr int kThreads = 128 * (kGroups + 2);
    static constexpr int kAux = kGroups, kIo = kGroups + 1;       // warpgroups of the other roles
    static constexpr int kQTile = 128 * D * 2;
    static constexpr int kTile = KT * D * 2;
    static constexpr int kHalf = KT * 128;                        // 64 columns of a tile
    static constexpr int kRawTile = KT * D, kRawRow = D == 64 ? 64 : 128;   // halves of 128-byte rows
    static constexpr int kRaw = kQuant ? kRawTile + 128 : 0;      // a raw stage: bytes and scales
    static constexpr int kRawStages = kQuant ? 4 : 0;
    static constexpr int kTail = kQuant ? 1536 : 2048;            // barriers and small arrays
    static constexpr int kBudget = 227 * 1024 - 1024 - kTail;
    static constexpr int kFit = (kBudget - kQTiles * kQTile - kRawStages * kRaw) / kTile;
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr int kSmem = 1024 + kQTiles * kQTile + kStages * kTile + kRawStages * kRaw + kTail;
    // TMEM columns
    static constexpr int kS = KT;                                  // per channel
    static constexpr int kO = D == 256 ? 128 : 256;                // first O column
    // the softmax keeps its row of S in registers from the maximum to P, or reads it again in
    // loops: next to the widening warps the longer code costs a third of the time in
    // instruction fetches (e4m3, d = 128: 776 against 888 TFLOP/s; bf16 1075 against 1051)
    static constexpr bool kHold = !kQuant;
    static constexpr int kParts = KT / 64;                         // P is handed over in parts of 64 keys
    static constexpr int kOStep = D;
    static_assert(kStages >= 3 && kSmem <= 227 * 1024, "tiles exceed shared memory");
};

// Ring order of an item's n tiles: K runs `lead` tiles ahead of V (0 for kRows, 1 otherwise).
// Position of K(j) and V(j) in that order.
template <int MODE>
__device__ __forceinline__ uint32_t seq_k(int j, int n) {
    if constexpr (MODE == kRows) return 2 * j;
    return j == 0 ? 0 : 2 * j - 1;
}
template <int MODE>
__device__ __forceinline__ uint32_t seq_v(int j, int n) {
    if constexpr (MODE == kRows) return 2 * j + 1;
    return min(j + 2, n) + j;
}
// The x-th tile in ring order: (is V, tile).
template <int MODE>
__device__ __forceinline__ void ring_tile(int x, int n, bool& v, int& j) {
    if constexpr (MODE == kRows) {
        v = x & 1;
        j = x >> 1;
    } else if (x == 0) {
        v = false;
        j = 0;
    } else if (x == 2 * n - 1) {
        v = true;
        j = n - 1;
    } else {
        v = !(x & 1);                 // K1 V0 K2 V1 ...
        j = v ? x / 2 - 1 : (x + 1) / 2;
    }
}

// Four e4m3 bytes -> two fp16 pairs, times the pair of factors.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t factor, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 s, t;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 s, l;\n\tcvt.rn.f16x2.e4m3x2 t, h;\n\t"
        "mul.rn.f16x2 %0, s, %3;\n\tmul.rn.f16x2 %1, t, %3;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w), "r"(factor));
}
template <bool kF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (kF16) {
        const __half2 p = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&p);
    } else {
        const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&p);
    }
}
template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int CD, int D, int MODE>
__global__ void __launch_bounds__(Tc<CD, D, MODE>::kThreads, 1)
k_paged_tc(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
           const __grid_constant__ PagedArgs a, int page_shift, uint64_t timeout_ns, int dbg) {
    using C = Tc<CD, D, MODE>;
    constexpr bool kQuant = C::kQuant;
    constexpr int KT = C::KT, NST = C::kStages, NRAW = C::kRawStages;
    constexpr uint32_t kExp = kQuant ? kExpF16 : kExpBf16;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    uint8_t* sQ = base;
    uint8_t* sT = sQ + C::kQTiles * C::kQTile;          // tile ring
    uint8_t* sR = sT + NST * C::kTile;                  // raw ring (e4m3)
    uint8_t* sScale = sR + NRAW * C::kRawTile;          // their scales, 128 bytes each
    uint64_t* full = reinterpret_cast<uint64_t*>(sScale + NRAW * 128);
    uint64_t* empty = full + 8;
    uint64_t* rfull = empty + 8;                        // e4m3: [4] raw tiles
    uint64_t* rempty = rfull + 4;
    uint64_t* cut_full = rfull;                         // else [8]: cut V tiles, by slot
    uint64_t* q_full = rempty + 4;                      // [2]
    uint64_t* s_full = q_full + 2;                      // [2] by channel
    uint64_t* p_full = s_full + 2;                      // [part][channel]
    uint64_t* o_full = p_full + 4;                      // kSingle: [0] after every P V
    uint64_t* o_last = o_full + 2;                      // kSingle: after the last P V of an item
    uint64_t* ml_ready = o_last + 1;
    uint64_t* merged = ml_ready + 1;
    uint64_t* mma_done = merged + 1;
    uint64_t* aux_done = mma_done + 1;                  // not e4m3: [8] cut V tiles are clean, by slot
    // forced timeouts: one that nothing arrives at in this mode
    uint64_t* never = MODE == kSingle ? &o_full[1] : o_last;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(aux_done + (kQuant ? 0 : 8));
    int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
    volatile int* odd = abort_flag + 1;                 // [16] by item: V had values taken out
    volatile uint32_t* unit = reinterpret_cast<volatile uint32_t*>(abort_flag + 17);   // [16] by ring position
    volatile uint32_t* gone = unit + 16;                // [16] 16-key groups without a page
    volatile uint32_t* r_other = gone + 16;             // kKeys: channel 1's R
    volatile float* ml = reinterpret_cast<volatile float*>(const_cast<uint32_t*>(r_other) + 1);   // [2][128]
    static_assert((kQuant ? 38 : 46) * 8 + 4 * (2 + 16 * 3 + 1 + 256) <= C::kTail, "small arrays");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = threadIdx.x >> 7;
    const int tid = threadIdx.x & 127;
    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            tc::mbar_init(&full[s], kQuant ? 128 : 1);
            tc::mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < NRAW; ++s) {
            tc::mbar_init(&rfull[s], 1);
            tc::mbar_init(&rempty[s], 128);
        }
        if (!kQuant)
            for (int s = 0; s < 8; ++s) {
                tc::mbar_init(&cut_full[s], 1);
                tc::mbar_init(&aux_done[s], 128);
            }
        for (int c = 0; c < 2; ++c) {
            tc::mbar_init(&q_full[c], 128);
            tc::mbar_init(&s_full[c], 1);
            tc::mbar_init(&p_full[c], 128);
            tc::mbar_init(&p_full[2 + c], 128);
            tc::mbar_init(&o_full[c], 1);
        }
        tc::mbar_init(ml_ready, 128);
        tc::mbar_init(merged, 128);
        tc::mbar_init(o_last, 1);
        tc::mbar_init(mma_done, 1);
        *abort_flag = 0;
        for (int i = 0; i < 16; ++i) {
            odd[i] = 0;
            unit[i] = 0;
            gone[i] = 0;
        }
        tc::fence_barrier_init();
    }
    if (warp == 0) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const tc::Guard gd{abort_flag, a.status, KID_PAGED_TC, timeout_ns};
    // A wait of a whole warp, which goes on or winds down together: what follows is collective.
    // (Once per tile and role where it costs: a vote behind every wait took 2 % of e4m3 chunks.  Until
    // the vote a failed wait's data is read, and nothing else.)
    auto warp_wait = [&](uint64_t* bar, uint32_t parity, int where) {
        return __all_sync(0xffffffffu, tc::wait(bar, parity, gd, where)) != 0;
    };
    const int G = a.Hq / a.kv.Hkv, Hkv = a.kv.Hkv;
    wait_for_previous();                       // the plan
    let_next_start();                          // the join may read the plan while this runs
    PagedWalk walk(a, blockIdx.x);
    PagedItem it;

    if (wg == C::kIo) {
        if constexpr (C::kGroups == 2) reg_dec<64>();
        if (warp == C::kIo * 4) {
            // ---------------- loader: one warp, one lane per page of a tile
            const int box = min(a.kv.page_size, KT);
            const int n_box = KT / box;
            uint32_t seq = 0;
            uint32_t n_cut = 0, was_cut = 0;         // by slot: parity of cut_full, last use
            bool ok = true;
            if (lane == 0) {
                tc::prefetch_tmap(&tmK);
                tc::prefetch_tmap(&tmV);
            }
            while (ok && walk.next(it)) {
                const int n = it.t1 - it.t0;
                const int pos_min = it.blk.pos0 + it.blk.row0 / G;
                for (int x = 0; ok && x < 2 * n; ++x, ++seq) {
                    bool v;
                    int j;
                    ring_tile<MODE>(x, n, v, j);
                    const int j0 = (it.t0 + j) * KT;
                    int id = -1, row = 0;
                    bool bad = false;
                    if (lane < n_box) {
                        const int key = j0 + lane * box;
                        row = key & (a.kv.page_size - 1);
                        if (key < it.blk.len) {
                            id = page_of(a.b, a.kv, it.blk.seq, page_shift, key, a.status, KID_PAGED_TC);
                            bad = id < 0;
                        }
                    }
                    // 16-key groups of the pages that are missing
                    uint32_t groups = 0;
                    const uint32_t bads = __ballot_sync(0xffffffffu, bad);
                    if (bads)
                        for (int p = 0; p < n_box; ++p)
                            if (bads >> p & 1) groups |= ((1u << (box / 16)) - 1) << (p * (box / 16));
                    const CUtensorMap* tm = v ? &tmV : &tmK;
                    if constexpr (!kQuant) {
                        const int s = seq % NST;
                        ok = warp_wait(&empty[s], ((seq / NST) & 1) ^ 1, 1);
                        if (!ok) break;
                        // a cut V tile goes to the auxiliary warps first, on a barrier of its
                        // own: the MMA issuer waits for theirs (aux_done)
                        const bool cut = v && j0 + KT - 1 > pos_min;
                        uint64_t* bar = cut ? &cut_full[s] : &full[s];
                        if (cut) {
                            n_cut ^= 1u << s;
                            was_cut |= 1u << s;
                        } else {
                            was_cut &= ~(1u << s);
                        }
                        if (lane == 0) {
                            gone[seq & 15] = groups;
                            tc::mbar_arrive_expect_tx(bar, C::kTile);
                            if (cut) tc::mbar_arrive(&full[s]);
                        }
                        __syncwarp();
                        if (lane < n_box)
                            for (int h = 0; h < D / 64; ++h)
                                tc::tma_load_4d(sT + s * C::kTile + h * C::kHalf + lane * box * 128, tm,
                                                bar, h * 64, row, it.g, id);
                    } else {
                        const int s = seq % NRAW;
                        ok = warp_wait(&rempty[s], ((seq / NRAW) & 1) ^ 1, 1);
                        if (!ok) break;
                        uint8_t* raw = sR + s * C::kRawTile;
                        uint8_t* sc = sScale + s * 128 + lane * box;
                        if (lane < n_box && id < 0) {
                            for (int i = 0; i < box; i += 4) *reinterpret_cast<uint32_t*>(sc + i) = 0;
                            tc::fence_proxy_async_smem();
                        }
                        const uint32_t have = __ballot_sync(0xffffffffu, lane < n_box && id >= 0);
                        __syncwarp();                         // the zeros come before the arrival
                        if (lane == 0) {
                            gone[seq & 15] = groups;
                            tc::mbar_arrive_expect_tx(&rfull[s], KT * D + __popc(have) * box);
                        }
                        __syncwarp();
                        if (lane < n_box) {
                            for (int h = 0; h < D / C::kRawRow; ++h)
                                tc::tma_load_4d(raw + h * KT * C::kRawRow + lane * box * C::kRawRow, tm,
                                                &rfull[s], h * C::kRawRow, row, it.g, id);
                            if (id >= 0)
                                tc::bulk_load(sc, (v ? a.kv.v_scale : a.kv.k_scale) +
                                                      (((int64_t)id * Hkv + it.g) << page_shift) + row,
                                              box, &rfull[s]);
                        }
                    }
                }
            }
            // the copies in flight land before the shared memory goes away
            int zero = 0;
            const tc::Guard drain{&zero, nullptr, 0, timeout_ns};
            constexpr int kRing = kQuant ? NRAW : NST;
            for (uint32_t s = seq > (uint32_t)kRing ? seq - kRing : 0; s < seq; ++s) {
                const uint32_t r = s % kRing;
                if (kQuant) tc::wait(&rfull[r], (s / kRing) & 1, drain, 0);
                else if (was_cut >> r & 1) tc::wait(&cut_full[r], (n_cut >> r & 1) ^ 1, drain, 0);
                else tc::wait(&full[r], (s / kRing) & 1, drain, 0);
            }
        } else if (warp == C::kIo * 4 + 1) {
            // ---------------- MMA issuer: the whole warp walks, one lane issues.  Everything the
            // walk depends on goes through a shuffle (tc::uniform): descriptors computed per
            // thread, or under a condition that could differ between threads, have to be moved to
            // uniform registers one by one, and the issue of the MMAs then takes longer than the
            // MMAs (d = 128: 804 instead of 1100 TFLOP/s).
            const bool lead = tc::elect_one();
            constexpr uint32_t idesc_s = kQuant ? tc::idesc_f16_f32(128, KT) : tc::idesc_bf16_f32(128, KT);
            constexpr uint32_t idesc_o = kQuant ? tc::idesc_f16_f32(128, D, false, true)
                                                : tc::idesc_bf16_f32(128, D, false, true);
            uint32_t seq0 = 0, nq[2] = {0, 0}, np[2] = {0, 0}, n_aux = 0;
            bool ok = true;
            auto tile_ready = [&](uint32_t s) {
                if (!warp_wait(&full[s % NST], (s / NST) & 1, 2)) return false;
                tc::fence_after_sync();
                return true;
            };
            const uint64_t dq = tc::uniform(tc::desc_kmajor_sw128(tc::smem_u32(sQ)));
            const uint64_t dk = tc::uniform(tc::desc_kmajor_sw128(tc::smem_u32(sT)));
            const uint64_t dv = tc::uniform(tc::desc_mnmajor_sw128(tc::smem_u32(sT), C::kHalf));
            const uint32_t ut = tc::uniform(tmem);
            auto commit = [&](uint64_t* bar) {
                if (lead) tc::mma_commit(bar);
            };
            auto issue_s = [&](int c, uint32_t s) {
                const uint32_t slot = tc::uniform(s % NST);
                const uint64_t a0 = dq + (MODE == kRows ? c : 0) * (C::kQTile >> 4);
                const uint64_t b0 = dk + slot * (C::kTile >> 4);
                if (lead) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        tc::mma_bf16_ss(ut + c * C::kS, a0 + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                                        b0 + (((kk >> 2) * C::kHalf + (kk & 3) * 32) >> 4), idesc_s,
                                        kk > 0 ? 1u : 0u);
                    tc::mma_commit(&s_full[c]);
                }
                __syncwarp();
            };
            // O += P V, part by part as the softmax warps hand P over
            auto issue_pv = [&](int c, uint32_t s, bool first) {
                const uint32_t slot = tc::uniform(s % NST);
                const uint64_t b0 = dv + slot * (C::kTile >> 4);
                const uint32_t o = ut + C::kO + (MODE == kSingle ? 0 : c) * C::kOStep;
                const uint32_t p = ut + c * C::kS;
                const uint32_t parity = np[c]++ & 1;
#pragma unroll
                for (int part = 0; part < C::kParts; ++part) {
                    if (!warp_wait(&p_full[2 * part + c], parity, 3)) return false;
                    tc::fence_after_sync();
                    if (lead) {
#pragma unroll
                        for (int kk = part * 4; kk < part * 4 + 4; ++kk)
                            tc::mma_f16_ts(o, p + kk * 8, b0 + ((kk * 16 * 128) >> 4), idesc_o,
                                           (!first || kk > 0) ? 1u : 0u);
                    }
                    __syncwarp();
                }
                return true;
            };
            while (ok && walk.next(it)) {
                const int n = (int)tc::uniform((uint32_t)(it.t1 - it.t0));
                const PagedBlock& k = it.blk;
                const bool two = MODE == kRows && tc::uniform((int64_t)k.n * G - k.row0 > 128 ? 1u : 0u) != 0;
                const int pos_min = (int)tc::uniform((uint32_t)(k.pos0 + k.row0 / G));
                const int t0 = (int)tc::uniform((uint32_t)it.t0);
                if (!(ok = warp_wait(&q_full[0], nq[0]++ & 1, 4))) break;
                if (two && !(ok = warp_wait(&q_full[1], nq[1]++ & 1, 4))) break;
                tc::fence_after_sync();
                auto v_ready = [&](int j) {
                    if (!tile_ready(seq0 + seq_v<MODE>(j, n))) return false;
                    if (!kQuant && (t0 + j) * KT + KT - 1 > pos_min) {
                        const uint32_t s = (seq0 + seq_v<MODE>(j, n)) % NST;
                        if (!warp_wait(&aux_done[s], n_aux >> s & 1, 5)) return false;
                        n_aux ^= 1u << s;
                        tc::fence_after_sync();
                    }
                    return true;
                };
                // kRows: both channels use every tile, in turns; otherwise tile j's channel (or,
                // kSingle, S buffer) alternates, one S ahead
                constexpr int kAhead = MODE == kRows ? 1 : 2;
                for (int j = 0; ok && j < min(kAhead, n); ++j) {
                    const uint32_t sk = seq0 + seq_k<MODE>(j, n);
                    if (!(ok = tile_ready(sk))) break;
                    issue_s(MODE == kRows ? 0 : j & 1, sk);
                    if (two) issue_s(1, sk);
                    commit(&empty[sk % NST]);
                }
                for (int j = 0; ok && j < n; ++j) {
                    const int c = MODE == kRows ? 0 : j & 1;
                    const bool more = j + kAhead < n;
                    const uint32_t sv = seq0 + seq_v<MODE>(j, n), sk = seq0 + seq_k<MODE>(j + kAhead, n);
                    // what can be waited for early is: P comes last
                    ok = v_ready(j) && (!more || tile_ready(sk)) &&
                         issue_pv(c, sv, MODE == kKeys ? j < 2 : j == 0);
                    if (!ok) break;
                    if (MODE == kSingle || !more) commit(&o_full[MODE == kSingle ? 0 : c]);
                    if (MODE == kSingle && j + 1 == n) commit(o_last);
                    if (!two) commit(&empty[sv % NST]);
                    if (more) {
                        issue_s(c, sk);
                        if (!two) commit(&empty[sk % NST]);
                    }
                    if (two) {
                        if (!(ok = issue_pv(1, sv, j == 0))) break;
                        commit(&empty[sv % NST]);
                        if (!more) {
                            commit(&o_full[1]);
                        } else {
                            issue_s(1, sk);
                            commit(&empty[sk % NST]);
                        }
                    }
                }
                seq0 += 2 * n;
            }
            commit(mma_done);
            int zero = 0;
            const tc::Guard drain{&zero, nullptr, 0, timeout_ns};
            tc::wait(mma_done, 0, drain, 0);
        }
    } else if (wg == C::kAux) {
        if constexpr (C::kGroups == 2) reg_dec<80>();
        // ---------------- widens e4m3 tiles; clears and cleans V where a tile is cut
        uint32_t seq = 0, item = 0, n_cut = 0;
        bool ok = true;
        while (ok && walk.next(it)) {
            const int n = it.t1 - it.t0;
            const PagedBlock& k = it.blk;
            const int pos_min = k.pos0 + k.row0 / G;
            uint32_t low = 255;                       // e4m3: scales of V, this thread's rows
            int high = 0;
            for (int x = 0; ok && x < 2 * n; ++x, ++seq) {
                bool v;
                int j;
                ring_tile<MODE>(x, n, v, j);
                const int j0 = (it.t0 + j) * KT;
                const bool cut = v && j0 + KT - 1 > pos_min;
                const int s = seq % NST;
                uint8_t* tile = sT + s * C::kTile;
                bool found = false;
                if constexpr (!kQuant) {
                    if (!cut) continue;
                    if (!(ok = warp_wait(&cut_full[s], n_cut >> s & 1, 6))) break;
                    n_cut ^= 1u << s;
                    constexpr int kVecs = C::kTile / 16 / 128;
#pragma unroll 4
                    for (int i = 0; i < kVecs; ++i) {
                        const int c = i * 128 + tid;                  // 16-byte chunk of the tile
                        const int row = (c >> 3) % KT;
                        uint4* p = reinterpret_cast<uint4*>(tile + c * 16);
                        uint4 w = *p;
                        const bool in = j0 + row < k.len;
                        const bool nf = not_finite2<kExp>(w.x) || not_finite2<kExp>(w.y) ||
                                        not_finite2<kExp>(w.z) || not_finite2<kExp>(w.w);
                        if (!in) {
                            *p = make_uint4(0, 0, 0, 0);
                        } else if (nf) {
                            found = true;
                            *p = make_uint4(finite_part<kExp>(w.x), finite_part<kExp>(w.y),
                                            finite_part<kExp>(w.z), finite_part<kExp>(w.w));
                        }
                    }
                    if (found) odd[item & 15] = 1;
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(&aux_done[s]);
                } else {
                    const int r = seq % NRAW;
                    ok = tc::wait(&rfull[r], (seq / NRAW) & 1, gd, 6);    // (voted on below)
                    // one thread per row (d = 256: two, a half each); the raw tile is swizzled by
                    // TMA, so that 8 rows read the same 16-byte column from different banks
                    const uint8_t* sc = sScale + r * 128;
                    const int row = tid % KT, hh = tid / KT;
                    const uint8_t* raw = sR + r * C::kRawTile + hh * KT * C::kRawRow + row * C::kRawRow;
                    const int rx = C::kRawRow == 64 ? (row >> 1) & 3 : row & 7;
                    // E: the largest scale of the tile's rows (0 = none, 255 = NaN left out)
                    uint32_t top = 0;
                    if (lane * 4 < KT) {
                        const uint32_t w = *reinterpret_cast<const uint32_t*>(sc + lane * 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t b = (w >> (8 * e)) & 255u;
                            if (b != kScaleNan && j0 + lane * 4 + e < k.len) top = max(top, b);
                        }
                    }
                    const int E = (int)__reduce_max_sync(0xffffffffu, top);
                    // 2^(e - E + 7) in fp16 (0 below 2^-24), NaN for a NaN scale
                    const uint32_t b = sc[row];
                    const bool in = j0 + row < k.len;
                    uint32_t f = 0;
                    if (in && b != 0) {
                        const int de = (int)b - E;
                        const __half h = __float2half_rn(b == kScaleNan ? __int_as_float(0x7fc00000)
                                                                        : pow2i(de + 7));
                        f = (uint32_t)__half_as_ushort(h) * 0x10001u;
                        // rows too far below the tile's largest, and the item's smallest scale of V
                        const bool far = de < (v ? -kSpan : -kExact);
                        if (far || b <= kScaleLeast) {
                            uint32_t any = 0;                 // a row of zeros does not count
                            for (int c = 0; c < C::kRawRow / 16; ++c) {
                                const uint4 w = *reinterpret_cast<const uint4*>(raw + (c << 4));
                                any |= w.x | w.y | w.z | w.w;
                            }
                            if (any & 0x7f7f7f7fu) {
                                if (far) mark_redo(a, it);
                                else if (v) low = min(low, b);
                            }
                        } else if (v) {
                            low = min(low, b);                // (NaN's is the largest)
                        }
                    }
                    if (v) high = max(high, E);
                    int tile_exp = E;
                    if (E <= (int)kScaleLeast) {              // perhaps zeros only: no exponent
                        constexpr int kRowVecs = C::kRawRow / 16;
                        uint32_t any = 0;
                        for (int c = lane; c < C::kRawTile / 16; c += 32)
                            if (j0 + c / kRowVecs % KT < k.len) {
                                const uint4 w = *reinterpret_cast<const uint4*>(sR + r * C::kRawTile + c * 16);
                                any |= (w.x | w.y | w.z | w.w) & 0x7f7f7f7fu;
                            }
                        if (!__any_sync(0xffffffffu, any != 0)) tile_exp = 0;
                    }
                    ok = tc::wait(&empty[s], ((seq / NST) & 1) ^ 1, gd, 7) && ok;
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    if (tid == 0) unit[seq & 15] = (uint32_t)tile_exp;
                    uint8_t* dst = tile + hh * 2 * C::kHalf + row * 128;
                    auto convert = [&](auto cut_tag) {
#pragma unroll 2
                        for (int c = 0; c < C::kRawRow / 16; ++c) {
                            const uint4 w = *reinterpret_cast<const uint4*>(raw + ((c ^ rx) << 4));
                            uint32_t y[8];
                            widen4(w.x, f, y[0], y[1]);
                            widen4(w.y, f, y[2], y[3]);
                            widen4(w.z, f, y[4], y[5]);
                            widen4(w.w, f, y[6], y[7]);
                            if constexpr (decltype(cut_tag)::value) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    found |= in && not_finite2<kExp>(y[e]);
                                    y[e] = in ? finite_part<kExp>(y[e]) : 0u;
                                }
                            }
                            uint8_t* d = dst + (c >> 2) * C::kHalf;
                            const int ch = (c & 3) * 2;
                            *reinterpret_cast<uint4*>(d + ((ch ^ (row & 7)) << 4)) =
                                make_uint4(y[0], y[1], y[2], y[3]);
                            *reinterpret_cast<uint4*>(d + (((ch + 1) ^ (row & 7)) << 4)) =
                                make_uint4(y[4], y[5], y[6], y[7]);
                        }
                    };
                    if (cut) convert(std::true_type{});
                    else convert(std::false_type{});
                    if (found) odd[item & 15] = 1;
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(&full[s]);
                    tc::mbar_arrive(&rempty[r]);
                }
            }
            if (kQuant && ok) {
                low = __reduce_min_sync(0xffffffffu, low);
                if (lane == 0 && high - (int)low > kSpan) mark_redo(a, it);
            }
            ++item;
        }
    } else {
        if constexpr (C::kGroups == 2) reg_inc<184>();
        // ---------------- softmax: thread = row = TMEM lane
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        uint32_t seq0 = 0, item = 0, ns[2] = {0, 0}, no = 0, n_ml = 0;
        bool ok = true;
        if (dbg & kDebugForceTimeout) ok = warp_wait(never, 0, 13);
        while (ok && walk.next(it)) {
            const int n = it.t1 - it.t0;
            const PagedBlock& k = it.blk;
            const int64_t rows_left = (int64_t)k.n * G - k.row0 - (MODE == kRows ? wg * 128 : 0);
            const uint32_t my_item = item++;
            const uint32_t my_seq = seq0;
            seq0 += 2 * n;
            if (MODE == kRows && wg == 1 && rows_left <= 0) continue;
            const int row = k.row0 + (MODE == kRows ? wg * 128 : 0) + tid;
            const bool valid = tid < rows_left;
            // the last key a row sees: the one at its position, or, of a length past the page table,
            // the last that the table has room for (what lies behind arrives as zeros)
            const int pos = valid ? min(k.pos0 + row / G, k.len - 1) : -1;
            const int pos_first = min(k.pos0 + (row - tid) / G, k.len - 1);
            const int64_t tok = k.tok0 + row / G;
            const int head = it.g * G + row % G;
            float fs = a.sl2;                         // scale of a raw score (log2 domain)
            if (MODE == kRows || wg == 0) {
                // this thread's row of Q, into the swizzled tile
                const uint4* src = reinterpret_cast<const uint4*>(
                    (const __nv_bfloat16*)a.q + ((valid ? tok : 0) * a.Hq + (valid ? head : 0)) * D);
                uint8_t* dst = sQ + (MODE == kRows ? wg : 0) * C::kQTile + tid * 128;
                float qs = 1.f;
                if constexpr (kQuant) {
                    uint32_t top = 0;
                    if (valid)
#pragma unroll 8
                        for (int c = 0; c < D / 8; ++c) {
                            const uint4 w = __ldg(src + c);
                            top = max(top, max(max(w.x & 0x7fffu, (w.x >> 16) & 0x7fffu),
                                               max(w.y & 0x7fffu, (w.y >> 16) & 0x7fffu)));
                            top = max(top, max(max(w.z & 0x7fffu, (w.z >> 16) & 0x7fffu),
                                               max(w.w & 0x7fffu, (w.w >> 16) & 0x7fffu)));
                        }
                    const int sh = min(14 - ((int)(top >> 7) - 127), 120);
                    qs = pow2i(sh);
                    fs = a.sl2 * pow2i(-sh);
                }
#pragma unroll 8
                for (int c = 0; c < D / 8; ++c) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (valid) w = __ldg(src + c);
                    if constexpr (kQuant) {
                        auto conv = [&](uint32_t y) {
                            return pack2<true>(__uint_as_float(y << 16) * qs,
                                               __uint_as_float(y & 0xffff0000u) * qs);
                        };
                        w = make_uint4(conv(w.x), conv(w.y), conv(w.z), conv(w.w));
                    }
                    *reinterpret_cast<uint4*>(dst + (c >> 3) * 16384 + (((c & 7) ^ (tid & 7)) << 4)) = w;
                }
                tc::fence_proxy_async_smem();
                tc::mbar_arrive(&q_full[MODE == kRows ? wg : 0]);
            }
            if (MODE == kKeys && kQuant && wg == 1) {
                // channel 1 scales its scores by channel 0's row factors
                uint32_t top = 0;
                const uint4* src = reinterpret_cast<const uint4*>(
                    (const __nv_bfloat16*)a.q + ((valid ? tok : 0) * a.Hq + (valid ? head : 0)) * D);
                if (valid)
#pragma unroll 8
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 w = __ldg(src + c);
                        top = max(top, max(max(w.x & 0x7fffu, (w.x >> 16) & 0x7fffu),
                                           max(w.y & 0x7fffu, (w.y >> 16) & 0x7fffu)));
                        top = max(top, max(max(w.z & 0x7fffu, (w.z >> 16) & 0x7fffu),
                                           max(w.w & 0x7fffu, (w.w >> 16) & 0x7fffu)));
                    }
                fs = a.sl2 * pow2i(-min(14 - ((int)(top >> 7) - 127), 120));
            }
            float m = -INFINITY, l = 0.f;
            int R = 0;                                // e4m3: running exponent of O's units
            const int j_first = MODE == kKeys ? wg : 0, j_step = MODE == kKeys ? 2 : 1;
            for (int j = j_first; ok && j < n; j += j_step) {
                const int c = MODE == kSingle ? (j & 1) : wg;
                const bool first = j == j_first;
                ok = tc::wait(&s_full[c], ns[c] & 1, gd, 8);      // (voted on below)
                ++ns[c];
                tc::fence_after_sync();
                const uint32_t ts = tmem + lanes + c * C::kS;
                const int j0 = (it.t0 + j) * KT;
                const uint32_t sk = my_seq + seq_k<MODE>(j, n);
                const uint32_t miss = gone[sk & 15];
                const bool masked = j0 + KT - 1 > pos_first || miss;
                // the row of S in parts of 64 columns
                float tm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                uint32_t hold[C::kHold ? C::kParts : 1][2][32];
                auto load_part = [&](uint32_t (&v)[2][32], int part) {
                    tc::tmem_ld32(ts + part * 64, v[0]);
                    tc::tmem_ld32(ts + part * 64 + 32, v[1]);
                };
                auto max_part = [&](uint32_t (&v)[2][32], int part) {
                    if (masked) {
                        const int lim = pos - j0 - part * 64;             // the last column seen
                        const uint32_t m4 = miss >> (part * 4);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (q * 32 + e > lim || (m4 >> ((q * 32 + e) / 16) & 1))
                                    v[q][e] = __float_as_uint(-INFINITY);
                            if (!C::kHold) tc::tmem_st32(ts + part * 64 + q * 32, v[q]);
                        }
                        if (!C::kHold) tc::tmem_wait_st();
                    }
#pragma unroll
                    for (int col = 0; col < 64; col += 2)
                        tm[(col >> 1) & 3] = tc::max3(tm[(col >> 1) & 3],
                                                      __uint_as_float(v[col / 32][col % 32]),
                                                      __uint_as_float(v[col / 32][col % 32 + 1]));
                };
                if constexpr (C::kHold) {
#pragma unroll
                    for (int part = 0; part < C::kParts; ++part) load_part(hold[part], part);
#pragma unroll
                    for (int part = 0; part < C::kParts; ++part) {
                        tc::tmem_wait_ld(hold[part][0]);
                        tc::tmem_wait_ld(hold[part][1]);
                    }
#pragma unroll
                    for (int part = 0; part < C::kParts; ++part) max_part(hold[part], part);
                } else {
#pragma unroll 1
                    for (int part = 0; part < C::kParts; ++part) {
                        load_part(hold[0], part);
                        tc::tmem_wait_ld(hold[0][0]);
                        tc::tmem_wait_ld(hold[0][1]);
                        max_part(hold[0], part);
                    }
                }
                float f = fs;
                int sh = 0;                           // P is stored times 2^sh
                float unit_corr = 1.f, unit_corr2 = 1.f;
                bool unit_move = false;
                if constexpr (kQuant) {
                    // above zero: masked scores are -inf here, and -inf * 0 is NaN (a zero row of Q
                    // over a tile of zero or missing rows of K: both factors are at their lowest)
                    f = fmaxf(fs * pow2i((int)unit[sk & 15] - 134), 0x1p-126f);
                    const uint32_t sv = my_seq + seq_v<MODE>(j, n);
                    ok = tc::wait(&full[sv % NST], (sv / NST) & 1, gd, 9) && ok;
                    int E = (int)unit[sv & 15];
                    if (E == 0) E = R ? R : 127;      // a tile without rows, or of zeros
                    if (first) R = E;
                    if (E > R || E + kSpread < R) {
                        unit_move = true;
                        unit_corr = pow2i((R - E) / 2);
                        unit_corr2 = pow2i(R - E - (R - E) / 2);
                        R = E;
                    }
                    sh = kBase + E - R;
                }
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const float tmax = fmaxf(fmaxf(tm[0], tm[1]), fmaxf(tm[2], tm[3])) * f;
                const bool raise = tmax > m + kLazy;
                const float m_new = raise ? tmax : m;
                const float corr = raise ? tc::ex2(m - m_new) : 1.f;
                if (!first && (__any_sync(0xffffffffu, raise) || unit_move)) {
                    // kSingle: O is shared by the two S buffers, the last P V may still run
                    if constexpr (MODE == kSingle)
                        if (!(ok = warp_wait(&o_full[0], (no + j - 1) & 1, 10))) break;
                    tc::fence_after_sync();
                    const uint32_t to = tmem + lanes + C::kO + (MODE == kSingle ? 0 : wg) * C::kOStep;
#pragma unroll 1
                    for (int q = 0; q < D / 16; ++q) {
                        uint32_t o[16];
                        tc::tmem_ld16(to + q * 16, o);
                        tc::tmem_wait_ld(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float y = __uint_as_float(o[e]) * corr;
                            if constexpr (kQuant) y = y * unit_corr * unit_corr2;
                            o[e] = __float_as_uint(y);
                        }
                        tc::tmem_st16(to + q * 16, o);
                    }
                    tc::tmem_wait_st();
                }
                m = m_new;
                // -m (0 for a row that has seen no key: its scores are -inf), plus P's exponent
                const float shift = (m_new == -INFINITY ? 0.f : -m_new) + (float)sh;
                const uint64_t f2 = tc::f2_pack(f, f), s2 = tc::f2_pack(shift, shift);
                uint64_t sum2[2] = {0ull, 0ull};
                auto exp_part = [&](uint32_t (&v)[2][32], int part) {
                    uint32_t w[32];
#pragma unroll
                    for (int col = 0; col < 64; col += 2) {
                        const uint64_t x2 = tc::f2_fma(
                            tc::f2_pack(__uint_as_float(v[col / 32][col % 32]),
                                        __uint_as_float(v[col / 32][col % 32 + 1])), f2, s2);
                        float x0, x1;
                        tc::f2_unpack(x2, x0, x1);
                        const float p0 = tc::ex2(x0), p1 = tc::ex2(x1);
                        sum2[(col >> 1) & 1] = tc::f2_add(sum2[(col >> 1) & 1], tc::f2_pack(p0, p1));
                        // P in 16 bits, the type of the product, two to a column
                        w[col / 2] = pack2<kQuant>(p0, p1);
                    }
                    // over columns of S that are read already
                    tc::tmem_st32(ts + part * 32, w);
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    tc::mbar_arrive(&p_full[2 * part + c]);
                };
                if constexpr (C::kHold) {
#pragma unroll
                    for (int part = 0; part < C::kParts; ++part) exp_part(hold[part], part);
                } else {
#pragma unroll 1
                    for (int part = 0; part < C::kParts; ++part) {
                        load_part(hold[0], part);
                        tc::tmem_wait_ld(hold[0][0]);
                        tc::tmem_wait_ld(hold[0][1]);
                        exp_part(hold[0], part);
                    }
                }
                float y0, y1, y2, y3;
                tc::f2_unpack(sum2[0], y0, y1);
                tc::f2_unpack(sum2[1], y2, y3);
                float sum = (y0 + y1) + (y2 + y3);
                if constexpr (kQuant) sum *= pow2i(-sh);
                l = l * corr + sum;
            }
            if (!ok) break;
            // ---- the item's result
            const int n_mine = MODE == kKeys ? (n - wg + 1) / 2 : n;
            if constexpr (MODE == kSingle) {
                // (o_full may be one or two phases behind here, which its parity cannot tell)
                ok = warp_wait(o_last, my_item & 1, 11);
                no += n;
            } else if (n_mine > 0) {
                ok = warp_wait(&o_full[wg], no++ & 1, 11);
            }
            if (!ok) break;
            tc::fence_after_sync();
            float w0 = 1.f, w1 = 0.f;                 // weights of the two channels' O
            if constexpr (kQuant) w0 = n_mine > 0 ? pow2i(R - 127) * 0x1p-15f : 0.f;
            bool other = false;
            if constexpr (MODE == kKeys) {
                if (wg == 1) {
                    ml[tid] = m;
                    ml[128 + tid] = l;
                    if (tid == 0) *r_other = (uint32_t)R;
                    tc::fence_before_sync();
                    tc::mbar_arrive(ml_ready);
                    if (!(ok = warp_wait(merged, n_ml++ & 1, 12))) break;
                    continue;
                }
                if (!(ok = warp_wait(ml_ready, n_ml++ & 1, 12))) break;
                tc::fence_after_sync();
                const float mb = ml[tid], lb = ml[128 + tid];
                other = n > 1;
                const float M = fmaxf(m, mb), ref = M == -INFINITY ? 0.f : M;
                const float fa = tc::ex2(m - ref), fb = other ? tc::ex2(mb - ref) : 0.f;
                w0 *= fa;
                w1 = fb;
                if constexpr (kQuant)
                    w1 *= other ? pow2i((int)*r_other - 127) * 0x1p-15f : 0.f;
                l = l * fa + (other ? lb * fb : 0.f);
                m = M;
            }
            const bool part = it.slot >= 0;
            const float inv = part ? 1.f : (l > 0.f || l != l ? 1.f / l : 0.f);
            const uint32_t to = tmem + lanes + C::kO + (MODE == kRows ? wg : 0) * C::kOStep;
            const int prow = (MODE == kRows ? wg * 128 : 0) + tid;
            float* ps = part ? part_slot(a, blockIdx.x, it.slot) : nullptr;
            const bool add_odd = odd[my_item & 15] != 0;
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
                __syncwarp();
                uint32_t o[32];
                tc::tmem_ld32(to + q * 32, o);
                tc::tmem_wait_ld(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * w0);
                if (MODE == kKeys && other) {
                    uint32_t o1[32];
                    tc::tmem_ld32(to + C::kOStep + q * 32, o1);
                    tc::tmem_wait_ld(o1);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = __float_as_uint(__uint_as_float(o[e]) + __uint_as_float(o1[e]) * w1);
                }
                if (add_odd && valid) {
                    // what was taken out of V in the cut tiles, for the keys this row sees
                    const int pos_min = k.pos0 + k.row0 / G;
                    const int last = min(pos, it.t1 * KT - 1);
                    for (int key = max(it.t0, max(pos_min, 0) / KT) * KT; key <= last; ++key) {
                        const int id = a.b.page_table[(int64_t)k.seq * a.b.max_pages + (key >> page_shift)];
                        if ((uint32_t)id >= (uint32_t)a.kv.n_pages) continue;
                        const int in = key & (a.kv.page_size - 1);
                        const int64_t at = id * a.kv.page_stride + in * a.kv.row_stride +
                                           it.g * a.kv.head_stride + q * 32;
                        const bool nan_row = kQuant &&
                            a.kv.v_scale[(((int64_t)id * Hkv + it.g) << page_shift) + in] == kScaleNan;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            float x;
                            if constexpr (kQuant) {
                                const uint32_t b = ((const uint8_t*)a.kv.v_pages)[at + e];
                                x = nan_row || (b & 127u) == 127u ? __int_as_float(0x7fc00000) : 0.f;
                            } else {
                                x = to_f(((const __nv_bfloat16*)a.kv.v_pages)[at + e]);
                            }
                            if (!isfinite(x)) o[e] = __float_as_uint(__uint_as_float(o[e]) + x);
                        }
                    }
                }
                if (valid && part) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<uint4*>(ps + (size_t)prow * D + q * 32 + e) =
                            make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                } else if (valid) {
                    __nv_bfloat16* orow = (__nv_bfloat16*)a.out + (tok * a.Hq + head) * D + q * 32;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            w[z] = pack2<false>(__uint_as_float(o[e + 2 * z]) * inv,
                                                __uint_as_float(o[e + 2 * z + 1]) * inv);
                        *reinterpret_cast<uint4*>(orow + e) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            if (valid && part) {
                ps[(size_t)C::kRb * D + prow] = m;
                ps[(size_t)C::kRb * (D + 1) + prow] = l;
            } else if (valid && a.lse) {
                a.lse[(int64_t)a.Hq * k.tok0 + (int64_t)head * k.n + row / G] = lse_of(m, l);
            }
            if (wg == 0 && tid == 0) odd[(my_item + 8) & 15] = 0;
            tc::fence_before_sync();
            if constexpr (MODE == kKeys) tc::mbar_arrive(merged);
        }
    }
    __syncthreads();
    if (warp == 0) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int CD, int D, int MODE>
cudaError_t launch(const PagedArgs& a, cudaStream_t st) {
    using C = Tc<CD, D, MODE>;
    CUtensorMap tk, tv;
    const uint64_t es = CD == TAM_E4M3 ? 1 : 2;
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)a.kv.page_size, (uint64_t)a.kv.Hkv,
                              (uint64_t)a.kv.n_pages};
    const uint64_t strides[3] = {a.kv.row_stride * es, a.kv.head_stride * es, a.kv.page_stride * es};
    const uint32_t rows = a.kv.page_size < C::KT ? a.kv.page_size : C::KT;
    const uint32_t boxes[4] = {CD == TAM_E4M3 ? (uint32_t)C::kRawRow : 64u, rows, 1, 1};
    if (!make_tmap_4d(&tk, CD == TAM_E4M3, a.kv.k_pages, dims, strides, boxes) ||
        !make_tmap_4d(&tv, CD == TAM_E4M3, a.kv.v_pages, dims, strides, boxes))
        return cudaErrorInvalidValue;
    auto kern = k_paged_tc<CD, D, MODE>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem((const void*)kern, C::kSmem, done);
    if (e != cudaSuccess) return e;
    int shift = 0;
    while ((1 << shift) < a.kv.page_size) ++shift;
    if ((e = launch_chained(kern, a.grid, C::kThreads, C::kSmem, st, tk, tv, a, shift, wait_timeout_ns(),
                            debug_flags())))
        return e;
    note_launch();
    return cudaSuccess;
}

// Applies fn.template operator()<CD, D, MODE>() for the call's shape: the rows of a sequence
// fill more than one tile of 128, or not.
template <class Fn>
auto by_shape(const PagedArgs& a, Fn fn) {
    const bool quant = a.kv.dtype == TAM_E4M3;
    const bool rows = (a.b.max_rows ? (int64_t)a.b.max_rows : a.T) * (a.Hq / a.kv.Hkv) > 128;
    switch (a.kv.d) {
        case 64:
            if (rows) return quant ? fn.template operator()<TAM_E4M3, 64, kRows>() : fn.template operator()<TAM_BF16, 64, kRows>();
            return quant ? fn.template operator()<TAM_E4M3, 64, kKeys>() : fn.template operator()<TAM_BF16, 64, kKeys>();
        case 128:
            if (rows) return quant ? fn.template operator()<TAM_E4M3, 128, kRows>() : fn.template operator()<TAM_BF16, 128, kRows>();
            return quant ? fn.template operator()<TAM_E4M3, 128, kKeys>() : fn.template operator()<TAM_BF16, 128, kKeys>();
        default:
            return quant ? fn.template operator()<TAM_E4M3, 256, kSingle>() : fn.template operator()<TAM_BF16, 256, kSingle>();
    }
}

// An item's own cost (Q, the first S, the output), in tiles of two channels: some 10 us.
// Ragged batch below: 902 us uncounted, 675 at 4, 617 at 6.
constexpr int kStart = 6;
struct ShapeOf {
    template <int CD, int D, int MODE>
    PagedShape operator()() const {
        return {Tc<CD, D, MODE>::kRb, Tc<CD, D, MODE>::KT, 148, kStart};
    }
};
struct Launch {
    const PagedArgs& a;
    cudaStream_t st;
    template <int CD, int D, int MODE>
    cudaError_t operator()() const { return launch<CD, D, MODE>(a, st); }
};

}  // namespace

PagedShape paged_tc_shape(const PagedArgs& a) { return by_shape(a, ShapeOf{}); }

cudaError_t paged_tc(const PagedArgs& a, cudaStream_t st) { return by_shape(a, Launch{a, st}); }

}  // namespace tam
