// Internal launcher interface of the paged KV cache: the arguments that tam_paged.cu hands
// to the kernels, and the workspace of the attention over pages.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>
#include <utility>

#include "../../include/tam.h"

namespace tam {

// A row block of the attention: RB consecutive (token, query head) rows of one sequence,
// which share every K/V tile of their KV head.  Row r of a sequence's n * G rows is query
// head r % G of the group at token r / G.  Written by the plan kernel.
struct PagedBlock {
    int32_t seq;
    int32_t row0;      // first row of the block
    int32_t nt;        // key tiles its last row sees (at least 1: an empty row is written too)
    int32_t tok0;      // first packed row of the sequence
    int32_t n;         // its new tokens (0 <= tok0, tok0 + n <= T)
    int32_t len;       // its keys (0 <= len <= capacity of its page-table row)
    int32_t pos0;      // position of its first new token (may be negative)
    int32_t pad;
    int64_t unit0;     // units of the blocks before this one (one KV head)
};

// Written by the plan kernel in front of the blocks.
struct PagedPlan {
    int32_t n_blocks;
    int32_t whole;     // 1: blocks are dealt whole, 0: the units are split evenly over the CTAs
    int32_t rest;      // split: the first `rest` CTAs take each + 1 of the units of all
    int32_t pad;       //        blocks and KV heads, the others `each`
    int64_t each;
};

struct PagedArgs {
    int64_t T;
    int Hq, dtype;
    const void* q;
    void* out;
    float* lse;
    tam_kv_cache kv;
    tam_paged_batch b;
    float sl2;                 // scale * log2(e)
    int32_t* status;
    // workspace
    PagedPlan* plan;
    PagedBlock* blocks;
    int max_blocks;            // blocks the plan can hold (never exceeded: see paged_max_blocks)
    float* part;               // partial results: 2 slots per CTA of part_floats(RB, d)
    int32_t* redo;             // 16-bit products over e4m3 pages, else NULL: [0] the number of
                               // items the join computes again, then a mark per item
                               // (kRedoMarks) and their list (kRedoMarks + redo_items)
    int64_t redo_items;        // max_blocks * Hkv
    int rb, kt, grid;          // rows per block, keys per tile, CTAs of the main kernel
    int start;                 // what an item costs besides its tiles, in tiles: an item (block,
                               // KV head) is start + nt units of work
};

// The plan keeps 20 bytes per sequence in shared memory.
constexpr int kMaxPlanSeqs = 8192;

constexpr int kRedoMarks = 64;

// One partial result: RB rows of O (fp32, unnormalised), then their maxima and sums.
inline __host__ __device__ size_t paged_part_floats(int rb, int d) { return (size_t)rb * (d + 2); }

// Upper bound of the blocks of a batch: every sequence may end inside one.
inline int64_t paged_max_blocks(int64_t T, int n_seq, int G, int rb) {
    return n_seq + (T * G) / rb + 1;
}

struct KvRowsArgs {
    int64_t T;
    int dtype;                 // of the packed rows
    void* k;                   // [T, Hkv, d]: read by the write, written by the read
    void* v;
    tam_kv_cache kv;
    tam_paged_batch b;
    int32_t* status;
};

cudaError_t kv_write(const KvRowsArgs& a, cudaStream_t st);
cudaError_t kv_read(const KvRowsArgs& a, cudaStream_t st);

// The three launches of a paged attention call: the plan (clears the status block), the
// main kernel, and the join of the blocks whose tiles were split.
cudaError_t paged_plan(const PagedArgs& a, cudaStream_t st);
cudaError_t paged_simt(const PagedArgs& a, cudaStream_t st);
cudaError_t paged_join(const PagedArgs& a, cudaStream_t st);

// Launches a kernel of the chain plan -> main -> join so that it may start while the kernel
// before it in the stream still runs (it waits with griddepcontrol before it reads anything
// that one writes): the launch latencies overlap.
template <class... Params, class... Args>
cudaError_t launch_chained(void (*kern)(Params...), unsigned grid, unsigned threads, size_t smem,
                           cudaStream_t st, Args&&... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// Sets a kernel's dynamic shared memory once per device (one `done` per kernel).
inline cudaError_t allow_smem(const void* kern, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Shapes of the main kernels: rows per block, keys per tile and CTAs.
struct PagedShape {
    int rb, kt, grid, start;
};
PagedShape paged_simt_shape(const PagedArgs& a);

// Chunks of rows: bf16 queries, tcgen05 on pages brought in by TMA.
PagedShape paged_tc_shape(const PagedArgs& a);
cudaError_t paged_tc(const PagedArgs& a, cudaStream_t st);

// Few rows per sequence (decoding): bf16 queries, mma.sync on streamed pages.
bool paged_few_supported(const PagedArgs& a);
PagedShape paged_few_shape(const PagedArgs& a);
cudaError_t paged_few(const PagedArgs& a, cudaStream_t st);

}  // namespace tam
