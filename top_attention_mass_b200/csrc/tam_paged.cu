// C ABI of the paged KV cache: argument checks, workspace layout and dispatch.
// Declarations and their contracts: include/tam.h.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "paged.h"

using namespace tam;

namespace {

constexpr int kMaxGroup = 128;
constexpr int kMaxKvHeads = 4096;

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? TAM_OK : TAM_ERR_CUDA; }

int elem_bytes(int dtype) { return dtype == TAM_F32 ? 4 : dtype == TAM_BF16 ? 2 : 1; }

int check_cache(const tam_kv_cache* kv) {
    if (!kv || !kv->k_pages || !kv->v_pages) return TAM_ERR_INVALID_ARG;
    if (kv->dtype != TAM_BF16 && kv->dtype != TAM_F32 && kv->dtype != TAM_E4M3)
        return TAM_ERR_INVALID_ARG;
    if (kv->n_pages < 1 || kv->Hkv < 1 || kv->page_size < 1) return TAM_ERR_INVALID_ARG;
    if (kv->d != 64 && kv->d != 128 && kv->d != 256) return TAM_ERR_UNSUPPORTED;
    if (kv->page_size < 16 || kv->page_size > 256 || (kv->page_size & (kv->page_size - 1)))
        return TAM_ERR_UNSUPPORTED;
    if (kv->n_pages >= (int64_t(1) << 31) || kv->Hkv > kMaxKvHeads) return TAM_ERR_UNSUPPORTED;
    const int64_t es = elem_bytes(kv->dtype);
    for (int64_t s : {kv->page_stride, kv->row_stride, kv->head_stride}) {
        if (s < kv->d || (s * es) % 16) return TAM_ERR_INVALID_ARG;
        if (s * es >= (int64_t(1) << 40)) return TAM_ERR_UNSUPPORTED;   // a tensor map's limit
    }
    if (!aligned16(kv->k_pages) || !aligned16(kv->v_pages)) return TAM_ERR_INVALID_ARG;
    if (kv->dtype == TAM_E4M3 && (!kv->k_scale || !kv->v_scale || !aligned16(kv->k_scale) ||
                                  !aligned16(kv->v_scale)))
        return TAM_ERR_INVALID_ARG;
    return TAM_OK;
}

int check_batch(const tam_kv_cache* kv, const tam_paged_batch* b, int64_t T) {
    if (!b || !b->page_table || !b->cu_rows || !b->kv_len) return TAM_ERR_INVALID_ARG;
    if (b->n_seq < 1 || b->max_pages < 1 || b->max_rows < 0 || T < 0) return TAM_ERR_INVALID_ARG;
    if (b->n_seq > kMaxPlanSeqs || T >= (int64_t(1) << 31) ||
        (int64_t)b->max_pages * kv->page_size > (int64_t(1) << 30))
        return TAM_ERR_UNSUPPORTED;
    return TAM_OK;
}

// The types of the packed rows a cache takes and gives.
int check_rows_dtype(const tam_kv_cache* kv, int dtype) {
    if (dtype != TAM_BF16 && dtype != TAM_F32) return TAM_ERR_INVALID_ARG;
    return kv->dtype == TAM_E4M3 || kv->dtype == dtype ? TAM_OK : TAM_ERR_UNSUPPORTED;
}

int move_rows(bool write, int64_t T, int dtype, void* k, void* v, const tam_kv_cache* kv,
              const tam_paged_batch* b, void* ws, size_t ws_bytes, void* stream) {
    int rc;
    if ((rc = check_cache(kv)) || (rc = check_batch(kv, b, T)) || (rc = check_rows_dtype(kv, dtype)))
        return rc;
    if (!ws || !aligned16(ws)) return TAM_ERR_INVALID_ARG;
    if (T > 0 && (!k || !v || !aligned16(k) || !aligned16(v))) return TAM_ERR_INVALID_ARG;
    if (ws_bytes < kStatusBytes) return TAM_ERR_WORKSPACE;
    cudaStream_t st = (cudaStream_t)stream;
    if ((rc = cuda_status(cudaMemsetAsync(ws, 0, kStatusBytes, st)))) return rc;
    if (T == 0) return TAM_OK;
    const KvRowsArgs a{T, dtype, k, v, *kv, *b, (int32_t*)ws};
    return cuda_status(write ? kv_write(a, st) : kv_read(a, st));
}

// Workspace: status block | plan | row blocks | partial results (2 per CTA) | items to be
// computed again.
struct PagedLayout {
    size_t off_plan, off_blocks, off_part, off_redo, total;
    int64_t max_blocks, redo_items;
    PagedShape shape;
    cudaError_t (*main)(const PagedArgs&, cudaStream_t);
};

int plan_layout(const PagedArgs& a, PagedLayout& p) {
    if (a.dtype == TAM_F32) {
        p.main = paged_simt;
        p.shape = paged_simt_shape(a);
    } else if (paged_few_supported(a)) {
        p.main = paged_few;
        p.shape = paged_few_shape(a);
    } else {
        p.main = paged_tc;
        p.shape = paged_tc_shape(a);
    }
    p.max_blocks = paged_max_blocks(a.T, a.b.n_seq, a.Hq / a.kv.Hkv, p.shape.rb);
    if (p.max_blocks >= (int64_t(1) << 31) - 1) return TAM_ERR_UNSUPPORTED;
    p.off_plan = kStatusBytes;
    p.off_blocks = p.off_plan + 256;
    p.off_part = p.off_blocks + align256((size_t)p.max_blocks * sizeof(PagedBlock));
    p.off_redo = p.off_part + align256((size_t)p.shape.grid * 2 * 4 * paged_part_floats(p.shape.rb, a.kv.d));
    p.redo_items = a.dtype == TAM_BF16 && a.kv.dtype == TAM_E4M3 ? p.max_blocks * a.kv.Hkv : 0;
    p.total = p.off_redo + (p.redo_items ? align256(4 * (kRedoMarks + 2 * (size_t)p.redo_items)) : 0);
    return TAM_OK;
}

int check_attention(int64_t T, int Hq, int dtype, const tam_kv_cache* kv, const tam_paged_batch* b) {
    int rc;
    if ((rc = check_cache(kv)) || (rc = check_batch(kv, b, T)) || (rc = check_rows_dtype(kv, dtype)))
        return rc;
    if (Hq < 1 || Hq % kv->Hkv != 0) return TAM_ERR_INVALID_ARG;
    if (Hq / kv->Hkv > kMaxGroup || T * Hq >= (int64_t(1) << 31)) return TAM_ERR_UNSUPPORTED;
    return TAM_OK;
}

PagedArgs shape_args(int64_t T, int Hq, int dtype, const tam_kv_cache* kv, const tam_paged_batch* b) {
    PagedArgs a{};
    a.T = T; a.Hq = Hq; a.dtype = dtype; a.kv = *kv; a.b = *b;
    a.sl2 = (float)(1.0 / std::sqrt((double)kv->d)) * kLog2e;
    return a;
}

}  // namespace

extern "C" {

int tam_kv_cache_write(int64_t T, int dtype, const void* k, const void* v, const tam_kv_cache* kv,
                       const tam_paged_batch* batch, void* workspace, size_t ws_bytes,
                       void* stream) {
    return move_rows(true, T, dtype, const_cast<void*>(k), const_cast<void*>(v), kv, batch,
                     workspace, ws_bytes, stream);
}

int tam_kv_cache_read(int64_t T, int dtype, void* k, void* v, const tam_kv_cache* kv,
                      const tam_paged_batch* batch, void* workspace, size_t ws_bytes,
                      void* stream) {
    return move_rows(false, T, dtype, k, v, kv, batch, workspace, ws_bytes, stream);
}

size_t tam_paged_attention_workspace(int64_t T, int Hq, int dtype, const tam_kv_cache* kv,
                                     const tam_paged_batch* batch) {
    if (check_attention(T, Hq, dtype, kv, batch) != TAM_OK) return 0;
    PagedLayout p{};
    if (plan_layout(shape_args(T, Hq, dtype, kv, batch), p) != TAM_OK) return 0;
    return p.total;
}

int tam_paged_gqa_attention(int64_t T, int Hq, int dtype, const void* q, const tam_kv_cache* kv,
                            const tam_paged_batch* batch, void* out, float* lse, void* workspace,
                            size_t ws_bytes, void* stream) {
    int rc = check_attention(T, Hq, dtype, kv, batch);
    if (rc) return rc;
    if (!workspace || !aligned16(workspace)) return TAM_ERR_INVALID_ARG;
    if (T > 0 && (!q || !out || !aligned16(q) || !aligned16(out) || (lse && !aligned16(lse))))
        return TAM_ERR_INVALID_ARG;
    PagedArgs a = shape_args(T, Hq, dtype, kv, batch);
    PagedLayout p{};
    if ((rc = plan_layout(a, p))) return rc;
    if (ws_bytes < p.total) return TAM_ERR_WORKSPACE;
    char* ws = (char*)workspace;
    a.q = q; a.out = out; a.lse = lse;
    a.status = (int32_t*)ws;
    a.plan = (PagedPlan*)(ws + p.off_plan);
    a.blocks = (PagedBlock*)(ws + p.off_blocks);
    a.part = (float*)(ws + p.off_part);
    a.redo_items = p.redo_items;
    a.redo = p.redo_items ? (int32_t*)(ws + p.off_redo) : nullptr;
    a.max_blocks = (int)p.max_blocks;
    a.rb = p.shape.rb; a.kt = p.shape.kt; a.grid = p.shape.grid;
    a.start = p.shape.start;
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) return cuda_status(cudaMemsetAsync(ws, 0, kStatusBytes, st));
    cudaError_t e = paged_plan(a, st);
    if (e == cudaSuccess) e = p.main(a, st);
    if (e == cudaSuccess) e = paged_join(a, st);
    return cuda_status(e);
}

}  // extern "C"
