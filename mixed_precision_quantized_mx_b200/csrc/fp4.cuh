// fp4.cuh -- geometry of microscaled 4-bit blobs as kernels see it, element types,
// and the launchers shared by the translation units of mx_fp4.h and mx_experts.h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mx_experts.h"
#include "mx_fp4.h"

namespace mx {
namespace fp4 {

constexpr int kRows = 128;                    // rows of a stored tile
constexpr int kCols = MX_FP4_KBLOCK;          // columns of a stored k-block
constexpr int kCodeBytes = kRows * kCols / 2; // 16 KB of codes per (tile, k-block)
constexpr int kMaxExperts = MX_EXPERTS_MAX;

// format constants: block columns, scale bytes of one (tile, k-block)
template <int FMT> struct Format;
template <> struct Format<MX_FP4_E4M3_16> { static constexpr int kBlock = 16; };
template <> struct Format<MX_FP4_E8M0_32> { static constexpr int kBlock = 32; };
template <int FMT> constexpr int scale_bytes() { return kRows * kCols / Format<FMT>::kBlock; }
template <int FMT> constexpr int tile_bytes() { return kCodeBytes + scale_bytes<FMT>(); }

// ---------------------------------------------------------------- element types
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// eight consecutive elements, 16-byte aligned, as fp32
__device__ __forceinline__ void load8v(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8v(const __half* p, float (&v)[8]) {
    const uint4 raw = *reinterpret_cast<const uint4*>(p);
    const __half2* h = reinterpret_cast<const __half2*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void load8v(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 raw = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void store8v(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8v(__half* p, const float (&v)[8]) {
    alignas(16) __half2 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(h);
}
__device__ __forceinline__ void store8v(__nv_bfloat16* p, const float (&v)[8]) {
    alignas(16) __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(h);
}

}  // namespace fp4

// ---------------------------------------------------------------- host side
// errors and pointer checks of the C boundary (mx_api.cu)
mx_status api_fail(mx_status st, const char* fmt, ...);
mx_status api_cuda_fail(cudaError_t e, const char* what);
// device (or managed) memory of the current device, else MX_ERR_INVALID_ARG
mx_status api_local_ptr(const void* p, const char* name);

inline int dtype_bytes(mx_dtype t) { return t == MX_F32 ? 4 : 2; }

// calls f with a null pointer of the element type
template <typename F> auto with_dtype(mx_dtype t, F f) {
    if (t == MX_F32) return f(static_cast<float*>(nullptr));
    if (t == MX_F16) return f(static_cast<__half*>(nullptr));
    return f(static_cast<__nv_bfloat16*>(nullptr));
}

// launches `kernel` on `s`; dependent = as a programmatic dependent of the kernel before it
template <typename... KArgs, typename... Args>
cudaError_t launch_ex(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster, bool dependent,
                      cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    int na = 0;
    if (cluster > 1) {
        at[na].id = cudaLaunchAttributeClusterDimension;
        at[na].val.clusterDim.x = cluster;
        at[na].val.clusterDim.y = 1;
        at[na].val.clusterDim.z = 1;
        ++na;
    }
    if (dependent) {
        at[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    cfg.attrs = at;
    cfg.numAttrs = na;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct PlanPtrs {
    int32_t *order, *pos, *dest, *offsets, *tiles;
};
inline PlanPtrs plan_ptrs(const mx_experts_layout& P, const void* plan) {
    uint8_t* b = const_cast<uint8_t*>(static_cast<const uint8_t*>(plan));
    auto at = [&](uint64_t o) { return reinterpret_cast<int32_t*>(b + o); };
    return {at(P.off_order), at(P.off_pos), at(P.off_dest), at(P.off_offsets), at(P.off_tiles)};
}

// fp4_quant.cu
cudaError_t launch_fp4_gscale(const mx_fp4_layout& L, const void* X, mx_dtype dt, int64_t ldx, int64_t gsx,
                              float* gscale, cudaStream_t s);
cudaError_t launch_fp4_quant(const mx_fp4_layout& L, const void* X, mx_dtype dt, int64_t ldx, int64_t gsx,
                             const float* gscale, void* blob, cudaStream_t s);
cudaError_t launch_fp4_quant_sorted(const mx_fp4_layout& L, const mx_experts_layout& P, const void* plan, bool sorted,
                                    const void* X, mx_dtype dt, int64_t ldx, const float* gscale, void* blob,
                                    bool early, cudaStream_t s);   // early: right behind the plan's sort
cudaError_t launch_fp4_dequant(const mx_fp4_layout& L, const void* blob, void* out, mx_dtype dt, int64_t ldo,
                               int64_t gso, cudaStream_t s);

// fp4_gemm.cu, fp4_stream.cu
struct Fp4Plan {
    int path;      // 1 stream, 2 pair
    int split;     // stream: CTAs per cluster
    int nt;        // stream: most tokens of a unit
    bool fused;    // the kernel can quantise the tokens itself
};
Fp4Plan fp4_gemm_plan(const mx_fp4_layout& LW, int M, const mx_experts_layout* P, const mx_fp4_opts* opts);

// tokens for the kernel to quantise (a fused plan)
struct Fp4Tokens {
    const void* X;
    mx_dtype dtype;
    int64_t ldx;
    const float* gscale;
    bool sorted;   // expert layer: rows of X are in sorted order
};
// M tokens, stored in ablob (LA) or raw in `tokens`.  P / plan NULL: one dense product.  early: the
// kernel before it in the stream is the quantiser that writes ablob.
cudaError_t launch_fp4_gemm(const mx_fp4_layout& LW, const void* wblob, int M, const mx_fp4_layout* LA,
                            const void* ablob, const Fp4Tokens* tokens, const mx_experts_layout* P, const void* plan,
                            void* Y, mx_dtype ydt, int64_t ldy, const mx_fp4_opts* opts, bool early, cudaStream_t s);

// experts.cu
cudaError_t launch_experts_sort(const mx_experts_layout& P, const int32_t* ids, void* plan, cudaStream_t s);
// the same by `ctas` CTAs (1, 2, 4, 8 or, where the device places such a cluster, 16); behind a first sort of the device
cudaError_t launch_experts_sort_on(const mx_experts_layout& P, const int32_t* ids, void* plan, int ctas, cudaStream_t s);
int sort_ctas(int n, bool wide);
cudaError_t launch_experts_gather(const mx_experts_layout& P, const void* plan, const void* X, mx_dtype dt, int H,
                                  int64_t ldx, void* Xs, int64_t lds, cudaStream_t s);
cudaError_t launch_experts_combine(const mx_experts_layout& P, const void* plan, const void* Ys, mx_dtype sdt, int H,
                                   int64_t lds, const float* w, void* Y, mx_dtype ydt, int64_t ldy, cudaStream_t s);
cudaError_t launch_experts_combine_bwd(const mx_experts_layout& P, const void* plan, const void* dY, const void* Ys,
                                       mx_dtype dt, int H, int64_t ldy, int64_t lds, const float* w, void* dYs,
                                       int64_t ldds, float* dw, cudaStream_t s);

}  // namespace mx
