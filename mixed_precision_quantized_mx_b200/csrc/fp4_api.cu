// fp4_api.cu -- the extern "C" boundary of mx_fp4.h and mx_experts.h: geometry,
// argument checks and the order of launches.
#include <cstring>

#include "fp4.cuh"

using mx::api_cuda_fail;
using mx::api_fail;
using mx::api_local_ptr;
using mx::dtype_bytes;

namespace {

uint64_t align256(uint64_t v) { return (v + 255) & ~uint64_t(255); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

#define MX_TRY(call)                                  \
    do {                                              \
        const mx_status st_ = (call);                 \
        if (st_ != MX_OK) return st_;                 \
    } while (0)

mx_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? MX_OK : api_cuda_fail(e, what); }

mx_status check_fp4(const mx_fp4_layout* L, const char* name) {
    if (L == nullptr) return api_fail(MX_ERR_INVALID_ARG, "%s is NULL", name);
    mx_fp4_layout ref;
    MX_TRY(mx_fp4_layout_init(L->rows, L->K, L->format, L->groups, &ref));
    if (memcmp(&ref, L, sizeof ref) != 0)
        return api_fail(MX_ERR_INVALID_ARG, "%s was modified after mx_fp4_layout_init", name);
    return MX_OK;
}

mx_status check_plan_layout(const mx_experts_layout* P) {
    if (P == nullptr) return api_fail(MX_ERR_INVALID_ARG, "experts layout is NULL");
    mx_experts_layout ref;
    MX_TRY(mx_experts_layout_init(P->T, P->k, P->E, &ref));
    if (memcmp(&ref, P, sizeof ref) != 0)
        return api_fail(MX_ERR_INVALID_ARG, "experts layout was modified after mx_experts_layout_init");
    return MX_OK;
}

// a buffer with sections: blob, plan or workspace
mx_status check_buffer(const void* p, const char* name) {
    MX_TRY(api_local_ptr(p, name));
    if (!aligned16(p)) return api_fail(MX_ERR_ALIGNMENT, "%s must be 16-byte aligned", name);
    return MX_OK;
}

mx_status check_dtype(mx_dtype t, const char* name) {
    if (t != MX_F32 && t != MX_F16 && t != MX_BF16) return api_fail(MX_ERR_INVALID_ARG, "bad %s %d", name, int(t));
    return MX_OK;
}

// a dense row-major matrix of `cols` columns with stride ld
mx_status check_rows(const void* p, const char* name, mx_dtype t, int cols, int64_t ld) {
    MX_TRY(check_dtype(t, "dtype"));
    if (ld < cols)
        return api_fail(MX_ERR_INVALID_ARG, "%s: row stride %lld < %d columns", name, (long long)ld, cols);
    MX_TRY(api_local_ptr(p, name));
    if (reinterpret_cast<uintptr_t>(p) % dtype_bytes(t) != 0)
        return api_fail(MX_ERR_ALIGNMENT, "%s is not aligned to its element", name);
    return MX_OK;
}

// fp32 or int32 vectors
mx_status check_vector(const void* p, const char* name) {
    MX_TRY(api_local_ptr(p, name));
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return api_fail(MX_ERR_ALIGNMENT, "%s is not aligned to its element", name);
    return MX_OK;
}

// the row kernels count the columns of a run of 1024 past the row's end in 32 bits
mx_status check_columns(int H) {
    if (H < 1) return api_fail(MX_ERR_INVALID_ARG, "H=%d", H);
    if (H > 0x7FFFFFFF - 1023) return api_fail(MX_ERR_UNSUPPORTED, "H=%d above 2^31 - 1024", H);
    return MX_OK;
}

mx_status check_gscale(const float* gscale, int format) {
    if (gscale == nullptr) return MX_OK;
    if (format == MX_FP4_E8M0_32)
        return api_fail(MX_ERR_INVALID_ARG, "the 32-column format has no matrix scale: gscale must be NULL");
    return check_vector(gscale, "gscale");
}

mx_status check_groups(const mx_fp4_layout* L, int64_t gs, const char* name) {
    if (L->groups > 1 && gs < 0) return api_fail(MX_ERR_INVALID_ARG, "%s: negative matrix stride", name);
    return MX_OK;
}

mx_status check_opts(const mx_fp4_opts* o, const mx_fp4_layout* LW) {
    if (o == nullptr) return MX_OK;
    if (o->path < 0 || o->path > 2) return api_fail(MX_ERR_INVALID_ARG, "path=%d (0, 1 or 2)", o->path);
    if (o->split != 0 && o->split != 1 && o->split != 2 && o->split != 4 && o->split != 8)
        return api_fail(MX_ERR_UNSUPPORTED, "split=%d (0, 1, 2, 4 or 8)", o->split);
    if (o->split > 1 && o->path == 2) return api_fail(MX_ERR_UNSUPPORTED, "path 2 does not split K");
    if (o->split > LW->kblocks)
        return api_fail(MX_ERR_UNSUPPORTED, "split=%d of %d k-blocks", o->split, LW->kblocks);
    if (o->wait_timeout_us < 0) return api_fail(MX_ERR_INVALID_ARG, "wait_timeout_us < 0");
    if (o->test_stall && !o->status) return api_fail(MX_ERR_INVALID_ARG, "test_stall needs a status word");
    if (o->status) MX_TRY(check_vector(o->status, "status"));
    return MX_OK;
}

mx_status check_weights(const mx_fp4_layout* LW, const void* wblob, int groups) {
    MX_TRY(check_fp4(LW, "weight layout"));
    if (LW->groups != groups)
        return api_fail(MX_ERR_INVALID_ARG, "weight layout holds %d matrices, %d expected", LW->groups, groups);
    if (LW->rows < 1) return api_fail(MX_ERR_INVALID_ARG, "weight layout has no rows");
    return check_buffer(wblob, "weight blob");
}

mx_status check_match(const mx_fp4_layout* LW, const mx_fp4_layout* LA) {
    MX_TRY(check_fp4(LA, "activation layout"));
    if (LA->groups != 1) return api_fail(MX_ERR_INVALID_ARG, "activation layout has %d groups", LA->groups);
    if (LA->K != LW->K || LA->format != LW->format)
        return api_fail(MX_ERR_INVALID_ARG, "weights have K=%d format %d, activations K=%d format %d", LW->K, LW->format,
                        LA->K, LA->format);
    return MX_OK;
}

mx_status sorted_layout(const mx_fp4_layout* LW, const mx_experts_layout* P, mx_fp4_layout* LA) {
    return mx_fp4_layout_init(P->max_rows, LW->K, LW->format, 1, LA);
}

mx_status check_linear_sorted(const mx_fp4_layout* LW, const void* wblob, const mx_experts_layout* P, const void* X,
                              mx_dtype xdtype, int64_t ldx, const float* gscale, const mx_fp4_opts* opts) {
    MX_TRY(check_weights(LW, wblob, P->E));
    MX_TRY(check_opts(opts, LW));
    MX_TRY(check_rows(X, "X", xdtype, LW->K, ldx));
    return check_gscale(gscale, LW->format);
}

// the launches of mx_fp4_linear_sorted, arguments checked
mx_status linear_sorted(const mx_fp4_layout* LW, const void* wblob, const mx_experts_layout* P, const void* plan,
                        bool sorted, const void* X, mx_dtype xdtype, int64_t ldx, const float* gscale, void* Y,
                        mx_dtype ydtype, int64_t ldy, void* workspace, const mx_fp4_opts* opts, bool early,
                        cudaStream_t s) {
    mx_fp4_layout LA;
    MX_TRY(sorted_layout(LW, P, &LA));
    if (mx::fp4_gemm_plan(*LW, LA.rows, P, opts).fused) {
        const mx::Fp4Tokens tokens{X, xdtype, ldx, gscale, sorted};
        return launched(mx::launch_fp4_gemm(*LW, wblob, LA.rows, nullptr, nullptr, &tokens, P, plan, Y, ydtype, ldy, opts,
                                            false, s),
                        "sorted fp4 linear launch");
    }
    MX_TRY(launched(mx::launch_fp4_quant_sorted(LA, *P, plan, sorted, X, xdtype, ldx, gscale, workspace, early, s),
                    "sorted fp4 quant launch"));
    return launched(mx::launch_fp4_gemm(*LW, wblob, LA.rows, &LA, workspace, nullptr, P, plan, Y, ydtype, ldy, opts, true,
                                        s),
                    "sorted fp4 GEMM launch");
}

}  // namespace

extern "C" {

mx_status mx_fp4_layout_init(int rows, int K, int format, int groups, mx_fp4_layout* out) {
    if (out == nullptr) return api_fail(MX_ERR_INVALID_ARG, "out is NULL");
    if (rows < 0 || K < 1 || groups < 1)
        return api_fail(MX_ERR_INVALID_ARG, "rows=%d K=%d groups=%d", rows, K, groups);
    if (format != MX_FP4_E4M3_16 && format != MX_FP4_E8M0_32)
        return api_fail(MX_ERR_UNSUPPORTED, "format=%d", format);
    if (K > (1 << 24)) return api_fail(MX_ERR_UNSUPPORTED, "K=%d above 2^24", K);
    mx_fp4_layout L;
    memset(&L, 0, sizeof L);
    L.rows = rows;
    L.K = K;
    L.format = format;
    L.groups = groups;
    L.block = format == MX_FP4_E4M3_16 ? 16 : 32;
    const int64_t tiles = (int64_t(rows) + mx::fp4::kRows - 1) / mx::fp4::kRows;
    if (tiles * groups * mx::fp4::kRows > 0x7FFFFFFF)
        return api_fail(MX_ERR_UNSUPPORTED, "rows=%d groups=%d: above 2^31 - 1 rows in all tiles", rows, groups);
    L.tiles = int32_t(tiles);
    L.kblocks = (K + MX_FP4_KBLOCK - 1) / MX_FP4_KBLOCK;
    L.tile_bytes = mx::fp4::kCodeBytes + mx::fp4::kRows * MX_FP4_KBLOCK / L.block;
    L.off_gscale = MX_HEADER_BYTES;
    L.off_data = align256(L.off_gscale + uint64_t(groups) * 4);
    L.total_bytes = L.off_data + uint64_t(groups) * L.tiles * L.kblocks * uint64_t(L.tile_bytes);
    *out = L;
    return MX_OK;
}

mx_status mx_fp4_layout_from_header(const void* host_header, size_t bytes, mx_fp4_layout* out) {
    if (host_header == nullptr || out == nullptr) return api_fail(MX_ERR_INVALID_ARG, "header or out is NULL");
    if (bytes < MX_HEADER_BYTES) return api_fail(MX_ERR_BAD_BLOB, "header shorter than %d bytes", MX_HEADER_BYTES);
    uint32_t h[6];
    memcpy(h, host_header, sizeof h);
    if (h[0] != MX_FP4_BLOB_MAGIC) return api_fail(MX_ERR_BAD_BLOB, "bad magic 0x%08x", h[0]);
    if (h[1] != MX_FP4_BLOB_VERSION)
        return api_fail(MX_ERR_BAD_BLOB, "blob version %u != %d", h[1], MX_FP4_BLOB_VERSION);
    if (mx_fp4_layout_init(int(h[2]), int(h[3]), int(h[4]), int(h[5]), out) != MX_OK)
        return api_fail(MX_ERR_BAD_BLOB, "header geometry invalid: rows=%d K=%d format=%d groups=%d", int(h[2]), int(h[3]),
                        int(h[4]), int(h[5]));
    return MX_OK;
}

mx_status mx_fp4_gscale(const mx_fp4_layout* L, const void* X, mx_dtype xdtype, int64_t ldx, int64_t gsx,
                        float* gscale, void* stream) {
    MX_TRY(check_fp4(L, "layout"));
    MX_TRY(check_groups(L, gsx, "X"));
    if (L->rows > 0) MX_TRY(check_rows(X, "X", xdtype, L->K, ldx));
    MX_TRY(check_vector(gscale, "gscale"));
    return launched(mx::launch_fp4_gscale(*L, X, xdtype, ldx, gsx, gscale, static_cast<cudaStream_t>(stream)),
                    "gscale launch");
}

mx_status mx_fp4_quant(const mx_fp4_layout* L, const void* X, mx_dtype xdtype, int64_t ldx, int64_t gsx,
                       const float* gscale, void* blob, void* stream) {
    MX_TRY(check_fp4(L, "layout"));
    MX_TRY(check_groups(L, gsx, "X"));
    if (L->rows > 0) MX_TRY(check_rows(X, "X", xdtype, L->K, ldx));
    else MX_TRY(check_dtype(xdtype, "dtype"));
    MX_TRY(check_gscale(gscale, L->format));
    MX_TRY(check_buffer(blob, "blob"));
    return launched(mx::launch_fp4_quant(*L, X, xdtype, ldx, gsx, gscale, blob, static_cast<cudaStream_t>(stream)),
                    "fp4 quant launch");
}

mx_status mx_fp4_quant_sorted(const mx_fp4_layout* L, const mx_experts_layout* P, const void* plan, int sorted,
                              const void* X, mx_dtype xdtype, int64_t ldx, const float* gscale, void* blob,
                              void* stream) {
    MX_TRY(check_fp4(L, "layout"));
    MX_TRY(check_plan_layout(P));
    if (L->groups != 1 || L->rows != P->max_rows)
        return api_fail(MX_ERR_INVALID_ARG, "layout has %d groups of %d rows, the plan takes one of %d", L->groups, L->rows,
                        P->max_rows);
    if (P->n > 0) MX_TRY(check_rows(X, "X", xdtype, L->K, ldx));
    else MX_TRY(check_dtype(xdtype, "dtype"));
    MX_TRY(check_gscale(gscale, L->format));
    MX_TRY(check_buffer(plan, "plan"));
    MX_TRY(check_buffer(blob, "blob"));
    return launched(mx::launch_fp4_quant_sorted(*L, *P, plan, sorted != 0, X, xdtype, ldx, gscale, blob, false,
                                                static_cast<cudaStream_t>(stream)),
                    "sorted fp4 quant launch");
}

mx_status mx_fp4_dequant(const mx_fp4_layout* L, const void* blob, void* out, mx_dtype odtype, int64_t ldo,
                         int64_t gso, void* stream) {
    MX_TRY(check_fp4(L, "layout"));
    MX_TRY(check_dtype(odtype, "dtype"));
    if (L->rows == 0) return MX_OK;
    MX_TRY(check_groups(L, gso, "out"));
    MX_TRY(check_buffer(blob, "blob"));
    MX_TRY(check_rows(out, "out", odtype, L->K, ldo));
    return launched(mx::launch_fp4_dequant(*L, blob, out, odtype, ldo, gso, static_cast<cudaStream_t>(stream)),
                    "fp4 dequant launch");
}

mx_status mx_fp4_gemm(const mx_fp4_layout* LW, const void* wblob, const mx_fp4_layout* LA, const void* ablob, void* Y,
                      mx_dtype ydtype, int64_t ldy, const mx_fp4_opts* opts, void* stream) {
    MX_TRY(check_fp4(LW, "weight layout"));
    MX_TRY(check_match(LW, LA));
    MX_TRY(check_dtype(ydtype, "dtype"));
    if (LA->rows == 0) return MX_OK;
    MX_TRY(check_weights(LW, wblob, 1));
    MX_TRY(check_opts(opts, LW));
    MX_TRY(check_buffer(ablob, "activation blob"));
    MX_TRY(check_rows(Y, "Y", ydtype, LW->rows, ldy));
    return launched(mx::launch_fp4_gemm(*LW, wblob, LA->rows, LA, ablob, nullptr, nullptr, nullptr, Y, ydtype, ldy, opts,
                                        false, static_cast<cudaStream_t>(stream)),
                    "fp4 GEMM launch");
}

mx_status mx_fp4_gemm_sorted(const mx_fp4_layout* LW, const void* wblob, const mx_fp4_layout* LA, const void* ablob,
                             const mx_experts_layout* P, const void* plan, void* Y, mx_dtype ydtype, int64_t ldy,
                             const mx_fp4_opts* opts, void* stream) {
    MX_TRY(check_fp4(LW, "weight layout"));
    MX_TRY(check_match(LW, LA));
    MX_TRY(check_plan_layout(P));
    MX_TRY(check_dtype(ydtype, "dtype"));
    if (P->n == 0) return MX_OK;
    MX_TRY(check_weights(LW, wblob, P->E));
    if (LA->rows != P->max_rows)
        return api_fail(MX_ERR_INVALID_ARG, "activation layout has %d rows, the plan takes %d", LA->rows, P->max_rows);
    MX_TRY(check_opts(opts, LW));
    MX_TRY(check_buffer(ablob, "activation blob"));
    MX_TRY(check_buffer(plan, "plan"));
    MX_TRY(check_rows(Y, "Y", ydtype, LW->rows, ldy));
    return launched(mx::launch_fp4_gemm(*LW, wblob, LA->rows, LA, ablob, nullptr, P, plan, Y, ydtype, ldy, opts, false,
                                        static_cast<cudaStream_t>(stream)),
                    "sorted fp4 GEMM launch");
}

mx_status mx_fp4_linear_workspace_size(const mx_fp4_layout* LW, int M, const mx_fp4_opts* opts, size_t* bytes) {
    MX_TRY(check_fp4(LW, "weight layout"));
    if (bytes == nullptr) return api_fail(MX_ERR_INVALID_ARG, "bytes is NULL");
    mx_fp4_layout LA;
    MX_TRY(mx_fp4_layout_init(M, LW->K, LW->format, 1, &LA));
    *bytes = M == 0 || mx::fp4_gemm_plan(*LW, M, nullptr, opts).fused ? 0 : LA.total_bytes;
    return MX_OK;
}

mx_status mx_fp4_linear(const mx_fp4_layout* LW, const void* wblob, const void* X, mx_dtype xdtype, int M, int64_t ldx,
                        const float* gscale, void* Y, mx_dtype ydtype, int64_t ldy, void* workspace, size_t ws_bytes,
                        const mx_fp4_opts* opts, void* stream) {
    MX_TRY(check_fp4(LW, "weight layout"));
    mx_fp4_layout LA;
    MX_TRY(mx_fp4_layout_init(M, LW->K, LW->format, 1, &LA));
    MX_TRY(check_dtype(xdtype, "xdtype"));
    MX_TRY(check_dtype(ydtype, "ydtype"));
    if (M == 0) return MX_OK;
    MX_TRY(check_weights(LW, wblob, 1));
    MX_TRY(check_opts(opts, LW));
    MX_TRY(check_rows(X, "X", xdtype, LW->K, ldx));
    MX_TRY(check_gscale(gscale, LW->format));
    MX_TRY(check_rows(Y, "Y", ydtype, LW->rows, ldy));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (mx::fp4_gemm_plan(*LW, M, nullptr, opts).fused) {
        const mx::Fp4Tokens tokens{X, xdtype, ldx, gscale, false};
        return launched(mx::launch_fp4_gemm(*LW, wblob, M, nullptr, nullptr, &tokens, nullptr, nullptr, Y, ydtype, ldy,
                                            opts, false, s),
                        "fp4 linear launch");
    }
    if (workspace == nullptr || ws_bytes < LA.total_bytes)
        return api_fail(MX_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", size_t(LA.total_bytes),
                        workspace ? ws_bytes : size_t(0));
    MX_TRY(check_buffer(workspace, "workspace"));
    MX_TRY(launched(mx::launch_fp4_quant(LA, X, xdtype, ldx, 0, gscale, workspace, s), "fp4 quant launch"));
    return launched(mx::launch_fp4_gemm(*LW, wblob, M, &LA, workspace, nullptr, nullptr, nullptr, Y, ydtype, ldy, opts,
                                        true, s),
                    "fp4 GEMM launch");
}

mx_status mx_fp4_linear_sorted_workspace_size(const mx_fp4_layout* LW, const mx_experts_layout* P,
                                              const mx_fp4_opts* opts, size_t* bytes) {
    MX_TRY(check_fp4(LW, "weight layout"));
    MX_TRY(check_plan_layout(P));
    if (bytes == nullptr) return api_fail(MX_ERR_INVALID_ARG, "bytes is NULL");
    mx_fp4_layout LA;
    MX_TRY(sorted_layout(LW, P, &LA));
    *bytes = P->n == 0 || mx::fp4_gemm_plan(*LW, LA.rows, P, opts).fused ? 0 : LA.total_bytes;
    return MX_OK;
}

mx_status mx_fp4_linear_sorted(const mx_fp4_layout* LW, const void* wblob, const mx_experts_layout* P,
                               const void* plan, int sorted, const void* X, mx_dtype xdtype, int64_t ldx,
                               const float* gscale, void* Y, mx_dtype ydtype, int64_t ldy, void* workspace,
                               size_t ws_bytes, const mx_fp4_opts* opts, void* stream) {
    size_t need = 0;
    MX_TRY(mx_fp4_linear_sorted_workspace_size(LW, P, opts, &need));
    MX_TRY(check_dtype(xdtype, "xdtype"));
    MX_TRY(check_dtype(ydtype, "ydtype"));
    if (P->n == 0) return MX_OK;
    MX_TRY(check_linear_sorted(LW, wblob, P, X, xdtype, ldx, gscale, opts));
    MX_TRY(check_buffer(plan, "plan"));
    MX_TRY(check_rows(Y, "Y", ydtype, LW->rows, ldy));
    if (need > 0) {
        if (workspace == nullptr || ws_bytes < need)
            return api_fail(MX_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                            workspace ? ws_bytes : size_t(0));
        MX_TRY(check_buffer(workspace, "workspace"));
    }
    return linear_sorted(LW, wblob, P, plan, sorted != 0, X, xdtype, ldx, gscale, Y, ydtype, ldy, workspace, opts,
                         false, static_cast<cudaStream_t>(stream));
}

mx_status mx_fp4_experts_workspace_size(const mx_fp4_layout* LW, const mx_experts_layout* P, const mx_fp4_opts* opts,
                                        size_t* bytes) {
    size_t act = 0;
    MX_TRY(mx_fp4_linear_sorted_workspace_size(LW, P, opts, &act));
    if (bytes == nullptr) return api_fail(MX_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = P->n == 0 ? 0 : P->total_bytes + align256(uint64_t(P->n) * LW->rows * 4) + act;
    return MX_OK;
}

mx_status mx_fp4_experts(const mx_fp4_layout* LW, const void* wblob, const mx_experts_layout* P, const int32_t* ids,
                         const void* X, mx_dtype xdtype, int64_t ldx, const float* gscale, const float* w, void* Y,
                         mx_dtype ydtype, int64_t ldy, void* workspace, size_t ws_bytes, const mx_fp4_opts* opts,
                         void* stream) {
    size_t need = 0;
    MX_TRY(mx_fp4_experts_workspace_size(LW, P, opts, &need));
    if (P->n == 0) return MX_OK;
    MX_TRY(check_columns(LW->rows));
    MX_TRY(check_vector(ids, "ids"));
    MX_TRY(check_vector(w, "w"));
    MX_TRY(check_rows(Y, "Y", ydtype, LW->rows, ldy));
    if (workspace == nullptr || ws_bytes < need)
        return api_fail(MX_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                        workspace ? ws_bytes : size_t(0));
    MX_TRY(check_buffer(workspace, "workspace"));
    uint8_t* const plan = static_cast<uint8_t*>(workspace);
    uint8_t* const ys = plan + P->total_bytes;
    const uint64_t act = P->total_bytes + align256(uint64_t(P->n) * LW->rows * 4);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // the product's checks come before the first launch: it is refused whole or not at all
    MX_TRY(check_linear_sorted(LW, wblob, P, X, xdtype, ldx, gscale, opts));
    MX_TRY(launched(mx::launch_experts_sort(*P, ids, plan, s), "experts sort launch"));
    MX_TRY(linear_sorted(LW, wblob, P, plan, false, X, xdtype, ldx, gscale, ys, MX_F32, LW->rows, plan + act, opts, true,
                         s));
    return launched(mx::launch_experts_combine(*P, plan, ys, MX_F32, LW->rows, LW->rows, w, Y, ydtype, ldy, s),
                    "experts combine launch");
}

// ---------------------------------------------------------------- experts
mx_status mx_experts_layout_init(int T, int k, int E, mx_experts_layout* out) {
    if (out == nullptr) return api_fail(MX_ERR_INVALID_ARG, "out is NULL");
    if (T < 0 || k < 1 || E < 1) return api_fail(MX_ERR_INVALID_ARG, "T=%d k=%d E=%d", T, k, E);
    if (E > MX_EXPERTS_MAX) return api_fail(MX_ERR_UNSUPPORTED, "E=%d above %d", E, MX_EXPERTS_MAX);
    const int64_t n = int64_t(T) * k;
    if (n > (1 << 24)) return api_fail(MX_ERR_UNSUPPORTED, "T=%d k=%d: above 2^24 slots", T, k);
    mx_experts_layout P;
    memset(&P, 0, sizeof P);
    P.T = T;
    P.k = k;
    P.E = E;
    P.n = int32_t(n);
    // every expert that has rows wastes at most 127 of its last tile
    const int64_t hit = n < E ? n : E;
    P.max_rows = int32_t((n + 127 * hit) / 128 * 128);
    uint64_t off = 0;
    P.off_order = off;   off = align256(off + uint64_t(n) * 4);
    P.off_pos = off;     off = align256(off + uint64_t(n) * 4);
    P.off_dest = off;    off = align256(off + uint64_t(n) * 4);
    P.off_offsets = off; off = align256(off + uint64_t(E + 1) * 4);
    P.off_tiles = off;   off = align256(off + uint64_t(E + 1) * 4);
    P.total_bytes = off;
    *out = P;
    return MX_OK;
}

mx_status mx_experts_sort(const mx_experts_layout* P, const int32_t* ids, void* plan, void* stream) {
    MX_TRY(check_plan_layout(P));
    if (P->n > 0) MX_TRY(check_vector(ids, "ids"));
    MX_TRY(check_buffer(plan, "plan"));
    return launched(mx::launch_experts_sort(*P, ids, plan, static_cast<cudaStream_t>(stream)), "experts sort launch");
}

mx_status mx_experts_gather(const mx_experts_layout* P, const void* plan, const void* X, mx_dtype dtype, int H,
                            int64_t ldx, void* Xs, int64_t lds, void* stream) {
    MX_TRY(check_plan_layout(P));
    MX_TRY(check_dtype(dtype, "dtype"));
    MX_TRY(check_columns(H));
    if (P->n == 0) return MX_OK;
    MX_TRY(check_buffer(plan, "plan"));
    MX_TRY(check_rows(X, "X", dtype, H, ldx));
    MX_TRY(check_rows(Xs, "Xs", dtype, H, lds));
    return launched(mx::launch_experts_gather(*P, plan, X, dtype, H, ldx, Xs, lds, static_cast<cudaStream_t>(stream)),
                    "experts gather launch");
}

mx_status mx_experts_gather_bwd(const mx_experts_layout* P, const void* plan, const void* dXs, mx_dtype dtype, int H,
                                int64_t lds, void* dX, int64_t ldx, void* stream) {
    MX_TRY(check_plan_layout(P));
    MX_TRY(check_dtype(dtype, "dtype"));
    MX_TRY(check_columns(H));
    if (P->n == 0) return MX_OK;
    MX_TRY(check_buffer(plan, "plan"));
    MX_TRY(check_rows(dXs, "dXs", dtype, H, lds));
    MX_TRY(check_rows(dX, "dX", dtype, H, ldx));
    return launched(mx::launch_experts_combine(*P, plan, dXs, dtype, H, lds, nullptr, dX, dtype, ldx,
                                               static_cast<cudaStream_t>(stream)),
                    "experts gather gradient launch");
}

mx_status mx_experts_combine(const mx_experts_layout* P, const void* plan, const void* Ys, mx_dtype sdtype, int H,
                             int64_t lds, const float* w, void* Y, mx_dtype ydtype, int64_t ldy, void* stream) {
    MX_TRY(check_plan_layout(P));
    MX_TRY(check_dtype(sdtype, "sdtype"));
    MX_TRY(check_dtype(ydtype, "ydtype"));
    MX_TRY(check_columns(H));
    if (P->n == 0) return MX_OK;
    MX_TRY(check_buffer(plan, "plan"));
    MX_TRY(check_rows(Ys, "Ys", sdtype, H, lds));
    MX_TRY(check_vector(w, "w"));
    MX_TRY(check_rows(Y, "Y", ydtype, H, ldy));
    return launched(mx::launch_experts_combine(*P, plan, Ys, sdtype, H, lds, w, Y, ydtype, ldy,
                                               static_cast<cudaStream_t>(stream)),
                    "experts combine launch");
}

mx_status mx_experts_combine_bwd(const mx_experts_layout* P, const void* plan, const void* dY, const void* Ys,
                                 mx_dtype dtype, int H, int64_t ldy, int64_t lds, const float* w, void* dYs,
                                 int64_t ldds, float* dw, void* stream) {
    MX_TRY(check_plan_layout(P));
    MX_TRY(check_dtype(dtype, "dtype"));
    MX_TRY(check_columns(H));
    if (P->n == 0) return MX_OK;
    MX_TRY(check_buffer(plan, "plan"));
    MX_TRY(check_rows(dY, "dY", dtype, H, ldy));
    MX_TRY(check_rows(Ys, "Ys", dtype, H, lds));
    MX_TRY(check_vector(w, "w"));
    MX_TRY(check_rows(dYs, "dYs", dtype, H, ldds));
    MX_TRY(check_vector(dw, "dw"));
    return launched(mx::launch_experts_combine_bwd(*P, plan, dY, Ys, dtype, H, ldy, lds, w, dYs, ldds, dw,
                                                   static_cast<cudaStream_t>(stream)),
                    "experts combine gradient launch");
}

}  // extern "C"
