// fp4_quant.cu -- microscaled 4-bit quantisation (E2M1 codes, one 8-bit scale per
// block of 16 or 32 columns), its inverse, and the matrix scale of the 16-column
// format.
//
// Quantiser: a thread holds 32 consecutive columns of a row, which is one or two blocks
// and one 16-byte chunk of stored codes; maxima come from its registers, so the
// matrix is read once.  A warp covers 1024 columns of one row, and lanes join their
// scale bytes into words.  The eight warps of a CTA take rows r, r+32, r+64, r+96, r+1,
// r+33, ..: the scale words of four such rows are neighbours in the stored tile and of
// eight fill a sector.  In front of an expert layer a token's row is quantised once and
// written to the places of all its slots.  Inverse: a thread holds eight columns, so that both its codes
// and its values are consecutive over a warp.  Both are bound by HBM: the matrix one way
// and 4.5 (or 4.25) bits a value the other.
#include "fp4_quant.cuh"

namespace mx {
namespace {

using namespace fp4;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The row of a matrix that a warp of row group rg (of rgs per tile) takes.  32-bit divisions, and
// none in the usual cases (64-bit ones cost the quantiser of 4096 x 8192 2.3 us).
struct Place {
    unsigned tile;       // of the blob
    int r;               // row in the tile
    int group, row;      // matrix and row in it
};
__device__ __forceinline__ Place place_of(unsigned rg, int rgs, int tiles, int warp) {
    Place p;
    const unsigned in = rgs == 16 ? rg & 15 : rg % unsigned(rgs);
    p.tile = rgs == 16 ? rg >> 4 : rg / unsigned(rgs);
    p.r = 2 * int(in) + (warp >> 2) + 32 * (warp & 3);
    p.group = tiles == 1 ? int(p.tile) : int(p.tile) < tiles ? 0 : int(p.tile / unsigned(tiles));
    p.row = int(p.tile - unsigned(p.group) * unsigned(tiles)) * kRows + p.r;
    return p;
}

struct QuantArgs {
    const void* X;
    int64_t ldx, gsx;
    const float* gscale;
    uint8_t* blob;
    uint64_t off_gscale, off_data;
    int rows, K, format, groups, tiles, kblocks;
    int segs;              // runs of 1024 columns per row
    int rgs;               // groups of eight rows per tile
    // expert order
    const int32_t *order, *dest;
    int n, k;
    int early;             // kTokens: the kernel before this one is the sort that writes the plan
};

// Which rows a kernel takes: matrices as they lie; rows in expert order, each to its place in the
// tiles; token rows, each to the places of all its slots (quantised once)
enum Rows { kMatrix, kSorted, kTokens };

// CTAs an SM holds at least, 16-column format: 16-bit types are bound by their arithmetic and gain from
// more warps (4096 x 8192: 17.7 us with five, 20.0 with four); fp32 fits four (26.4 us, three 29.4).  The
// 32-column format, with less arithmetic, needs no bound.
template <typename T, int FMT> constexpr int kQuantBlocks = FMT != MX_FP4_E4M3_16 ? 1 : sizeof(T) == 2 ? 5 : 4;

__device__ __forceinline__ void begin() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
}

template <typename T, int FMT, bool ALIGNED, int ROWS>
__global__ void __launch_bounds__(kThreads, kQuantBlocks<T, FMT>) fp4_quant_kernel(const __grid_constant__ QuantArgs a) {
    // The kernel before this one may still write X; the product after it may start streaming its
    // weights.  Behind its own sort, which lets it launch only after the sort's wait, X is complete and
    // the plan is not: the row is quantised first and the wait comes before anything is written
    // (2048 tokens of 4 of 64 experts, the whole layer: 67.5 -> 66.2 us).
    const bool late = ROWS == kTokens && a.early;
    if (!late) begin();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto header = [&] {
        if (blockIdx.x != 0) return;
        if (threadIdx.x < MX_HEADER_BYTES / 4) {
            const uint32_t h[6] = {MX_FP4_BLOB_MAGIC, MX_FP4_BLOB_VERSION, uint32_t(a.rows),
                                   uint32_t(a.K),     uint32_t(a.format),  uint32_t(a.groups)};
            uint32_t w = 0;
#pragma unroll
            for (int i = 0; i < 6; ++i) w = int(threadIdx.x) == i ? h[i] : w;
            reinterpret_cast<uint32_t*>(a.blob)[threadIdx.x] = w;
        }
        for (int i = threadIdx.x; i < a.groups; i += kThreads)
            reinterpret_cast<float*>(a.blob + a.off_gscale)[i] = a.gscale ? a.gscale[i] : 1.0f;
    };
    if (!late) header();
    // this warp's row and its 1024 columns
    const int seg = int(blockIdx.x % unsigned(a.segs));
    const unsigned rg = blockIdx.x / unsigned(a.segs);
    const T* row;
    int64_t tile_row = 0;                          // row of the blob's tiles (kMatrix, kSorted)
    float g = 1.0f;
    if constexpr (ROWS == kMatrix) {
        const Place at = place_of(rg, a.rgs, a.tiles, warp);
        const int grp = at.group, row_in = at.row;
        if (row_in >= a.rows) return;
        tile_row = int64_t(at.tile) * kRows + at.r;
        row = static_cast<const T*>(a.X) + int64_t(grp) * a.gsx + int64_t(row_in) * a.ldx;
        if (a.gscale) g = a.gscale[grp];
    } else {
        const int64_t p = int64_t(rg) * kWarps + warp;
        if (p >= a.n) {
            if (late) {
                begin();
                header();
            }
            return;
        }
        if (ROWS == kSorted) {
            const int slot = a.order[p];
            if (slot < 0) return;
            tile_row = a.dest[slot];
        }
        row = static_cast<const T*>(a.X) + p * a.ldx;
        if (a.gscale) g = a.gscale[0];
    }
    const int ch = seg * 32 + lane;                // 32-column chunk of the row
    const bool live = ch < a.kblocks * (kCols / 32);
    const int kb = ch >> 3, ci = ch & 7;
    uint32_t sb = 0, codes[4] = {};
    Columns<T> x;
    if constexpr (ALIGNED && sizeof(T) == 4) {
        // a lane's 32 columns are a whole line, which its eight loads would fetch a piece at a time; the
        // warp loads its 4 KB in order and exchanges them through shared memory (4096 x 8192: 26.3 us, 35.3
        // without)
        __shared__ uint4 line[kWarps][256];
        uint4* const own = line[warp];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = lane + 32 * j, col = seg * 1024 + 4 * c;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (col + 4 <= a.K) {
                v = *reinterpret_cast<const uint4*>(row + col);
            } else {
                if (col < a.K) v.x = __float_as_uint(row[col]);
                if (col + 1 < a.K) v.y = __float_as_uint(row[col + 1]);
                if (col + 2 < a.K) v.z = __float_as_uint(row[col + 2]);
            }
            own[c ^ ((c >> 3) & 7)] = v;
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) reinterpret_cast<uint4*>(x.w)[j] = own[8 * lane + (j ^ (lane & 7))];
    } else if (live) {
        x.template load<ALIGNED>(row, ch * 32, a.K);
    }
    if (live) sb = quant_columns<FMT>(x, matrix_scale(g), codes);
    // scale bytes of two (or four) lanes are one word of the stored section
    uint32_t word;
    bool writes;
    int at;
    if constexpr (FMT == MX_FP4_E4M3_16) {
        word = (sb << (16 * (lane & 1))) | (__shfl_xor_sync(0xffffffffu, sb, 1) << (16 * (~lane & 1)));
        writes = live && (lane & 1) == 0;
        at = 512 * (ci >> 1);
    } else {
        word = sb << (8 * (lane & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 1);
        word |= __shfl_xor_sync(0xffffffffu, word, 2);
        writes = live && (lane & 3) == 0;
        at = 512 * (ci >> 2);
    }
    auto put = [&](int64_t to) {
        const int r = int(to % kRows);
        uint8_t* const t = a.blob + a.off_data + (uint64_t(to / kRows) * a.kblocks + kb) * tile_bytes<FMT>();
        if (live)
            *reinterpret_cast<uint4*>(t + r * 128 + ((ci ^ (r & 7)) << 4)) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
        if (writes) *reinterpret_cast<uint32_t*>(t + kCodeBytes + at + 16 * (r & 31) + 4 * (r >> 5)) = word;
    };
    if constexpr (ROWS == kTokens) {
        if (late) {
            begin();
            header();
        }
        int mine = -1;                             // lane j's slot's row, -1 where dropped
        for (int j = 0; j < a.k; ++j) {
            if ((j & 31) == 0) {                   // the places of 32 slots
                const int64_t p = int64_t(rg) * kWarps + warp;
                mine = j + lane < a.k ? a.dest[p * a.k + j + lane] : -1;
            }
            const int to = __shfl_sync(0xffffffffu, mine, j & 31);
            if (to >= 0) put(to);
        }
    } else {
        put(tile_row);
    }
}

// ---------------------------------------------------------------- the inverse
struct DequantArgs {
    const uint8_t* blob;
    uint64_t off_gscale, off_data;
    void* out;
    int64_t ldo, gso;
    int rows, K, tiles, kblocks, segs, rgs;
};

// eight codes as fp32 (exact)
__device__ __forceinline__ void e2m1_values(uint32_t w, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

constexpr int kDeqIter = 4;                        // k-blocks that a warp takes together

template <typename T, int FMT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) fp4_dequant_kernel(const __grid_constant__ DequantArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kBlock = Format<FMT>::kBlock;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int seg = int(blockIdx.x % unsigned(a.segs));
    const Place at = place_of(blockIdx.x / unsigned(a.segs), a.rgs, a.tiles, warp);
    const int grp = at.group, r = at.r, row_in = at.row;
    const int64_t tile = at.tile;
    if (row_in >= a.rows) return;
    // lane: columns 8 lane .. 8 lane + 7 of each k-block, a word of chunk lane / 4
    const int bi = lane * 8 / kBlock, kb0 = seg * kDeqIter;
    const uint8_t* const t = a.blob + a.off_data + (uint64_t(tile) * a.kblocks + kb0) * tile_bytes<FMT>();
    const int code_at = r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4;
    const int scale_at = kCodeBytes + 512 * (bi >> 2) + 16 * (r & 31) + 4 * (r >> 5) + (bi & 3);
    const float g = reinterpret_cast<const float*>(a.blob + a.off_gscale)[grp];
    uint32_t w[kDeqIter], sb[kDeqIter];
#pragma unroll
    for (int i = 0; i < kDeqIter; ++i) {
        if (kb0 + i < a.kblocks) {
            w[i] = *reinterpret_cast<const uint32_t*>(t + i * tile_bytes<FMT>() + code_at);
            sb[i] = t[i * tile_bytes<FMT>() + scale_at];
        }
    }
    T* const o = static_cast<T*>(a.out) + int64_t(grp) * a.gso + int64_t(row_in) * a.ldo;
#pragma unroll
    for (int i = 0; i < kDeqIter; ++i) {
        const int c = (kb0 + i) * kCols + lane * 8;
        if (c >= a.K) break;
        const float s = FMT == MX_FP4_E4M3_16 ? e4m3_value(sb[i]) : e8m0_value(sb[i]);
        float v[8];
        e2m1_values(w[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(__fmul_rn(v[j], s), g);
        if (ALIGNED && c + 8 <= a.K) {
            store8v(o + c, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < a.K) o[c + j] = from_f32<T>(v[j]);
        }
    }
}

// ---------------------------------------------------------------- the matrix scale
// gscale first collects the largest finite |x| as integer bits (atomicMax of whole
// numbers: the order does not matter), then becomes the scale.
template <typename T>
__global__ void __launch_bounds__(kThreads)
fp4_amax_kernel(const T* X, int64_t ldx, int64_t gsx, int rows, int K, uint32_t* amax) {
    const T* x = X + int64_t(blockIdx.y) * gsx;
    uint32_t m = 0;
    // unsigned: the last step goes past the rows, of which there may be 2^31 - 128
    for (unsigned r = blockIdx.x * kWarps + (threadIdx.x >> 5); r < unsigned(rows); r += gridDim.x * kWarps) {
        const T* row = x + int64_t(r) * ldx;
#pragma unroll 8
        for (int c = threadIdx.x & 31; c < K; c += 32) {
            const uint32_t b = __float_as_uint(to_f32(row[c])) & 0x7FFFFFFFu;
            if (b < kInfBits) m = max(m, b);
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0 && m) atomicMax(amax + blockIdx.y, m);
}

__global__ void fp4_gscale_kernel(float* gscale, int groups) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= groups) return;
    const float q = __fdiv_rn(gscale[i], 2688.0f);            // 6 * 448
    gscale[i] = q >= 7.888609052210118e-31f ? q : 1.0f;       // 2^-100
}

bool rows_aligned(const void* p, int64_t ld, int64_t gs, int esz) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * esz) % 16 == 0 && (gs * esz) % 16 == 0;
}

template <int ROWS>
cudaError_t quant_launch(const QuantArgs& a, mx_dtype dt, bool aligned, int64_t blocks, cudaStream_t s) {
    return with_dtype(dt, [&](auto* tp) {
        using T = std::remove_pointer_t<decltype(tp)>;
        auto k = a.format == MX_FP4_E4M3_16
                     ? (aligned ? fp4_quant_kernel<T, MX_FP4_E4M3_16, true, ROWS>
                                : fp4_quant_kernel<T, MX_FP4_E4M3_16, false, ROWS>)
                     : (aligned ? fp4_quant_kernel<T, MX_FP4_E8M0_32, true, ROWS>
                                : fp4_quant_kernel<T, MX_FP4_E8M0_32, false, ROWS>);
        return launch_ex(k, dim3(unsigned(blocks)), dim3(kThreads), 0, 1, true, s, a);
    });
}

// runs of 1024 columns (four k-blocks) per row
int segs_of(const mx_fp4_layout& L) { return (L.kblocks + 3) / 4; }

// groups of eight rows per tile: 16, or what a single short tile has
int rgs_of(const mx_fp4_layout& L) { return L.rows >= 32 ? 16 : (L.rows + 1) / 2; }

QuantArgs quant_args(const mx_fp4_layout& L, const void* X, int64_t ldx, int64_t gsx, const float* gscale, void* blob) {
    QuantArgs a{};
    a.X = X;
    a.ldx = ldx;
    a.gsx = gsx;
    a.gscale = gscale;
    a.blob = static_cast<uint8_t*>(blob);
    a.off_gscale = L.off_gscale;
    a.off_data = L.off_data;
    a.rows = L.rows;
    a.K = L.K;
    a.format = L.format;
    a.groups = L.groups;
    a.tiles = L.tiles;
    a.kblocks = L.kblocks;
    a.segs = segs_of(L);
    return a;
}

}  // namespace

cudaError_t launch_fp4_quant(const mx_fp4_layout& L, const void* X, mx_dtype dt, int64_t ldx, int64_t gsx,
                             const float* gscale, void* blob, cudaStream_t s) {
    QuantArgs a = quant_args(L, X, ldx, gsx, gscale, blob);
    a.rgs = rgs_of(L) > 0 ? rgs_of(L) : 1;
    const int64_t blocks = int64_t(L.groups) * L.tiles * a.rgs * a.segs;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return quant_launch<kMatrix>(a, dt, rows_aligned(X, ldx, L.groups > 1 ? gsx : 0, dtype_bytes(dt)),
                               blocks > 0 ? blocks : 1, s);
}

cudaError_t launch_fp4_quant_sorted(const mx_fp4_layout& L, const mx_experts_layout& P, const void* plan, bool sorted,
                                    const void* X, mx_dtype dt, int64_t ldx, const float* gscale, void* blob,
                                    bool early, cudaStream_t s) {
    QuantArgs a = quant_args(L, X, ldx, 0, gscale, blob);
    a.early = early;
    const PlanPtrs pp = plan_ptrs(P, plan);
    a.order = pp.order;
    a.dest = pp.dest;
    a.n = sorted ? P.n : P.T;
    a.k = P.k;
    const int64_t blocks = int64_t((a.n + kWarps - 1) / kWarps) * a.segs;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const bool aligned = rows_aligned(X, ldx, 0, dtype_bytes(dt));
    return sorted ? quant_launch<kSorted>(a, dt, aligned, blocks > 0 ? blocks : 1, s)
                  : quant_launch<kTokens>(a, dt, aligned, blocks > 0 ? blocks : 1, s);
}

cudaError_t launch_fp4_dequant(const mx_fp4_layout& L, const void* blob, void* out, mx_dtype dt, int64_t ldo,
                               int64_t gso, cudaStream_t s) {
    DequantArgs a{};
    a.blob = static_cast<const uint8_t*>(blob);
    a.off_gscale = L.off_gscale;
    a.off_data = L.off_data;
    a.out = out;
    a.ldo = ldo;
    a.gso = gso;
    a.rows = L.rows;
    a.K = L.K;
    a.tiles = L.tiles;
    a.kblocks = L.kblocks;
    a.segs = segs_of(L);
    a.rgs = rgs_of(L);
    const int64_t blocks = int64_t(L.groups) * L.tiles * a.rgs * a.segs;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const bool aligned = rows_aligned(out, ldo, L.groups > 1 ? gso : 0, dtype_bytes(dt));
    return with_dtype(dt, [&](auto* tp) {
        using T = std::remove_pointer_t<decltype(tp)>;
        auto k = L.format == MX_FP4_E4M3_16
                     ? (aligned ? fp4_dequant_kernel<T, MX_FP4_E4M3_16, true> : fp4_dequant_kernel<T, MX_FP4_E4M3_16, false>)
                     : (aligned ? fp4_dequant_kernel<T, MX_FP4_E8M0_32, true> : fp4_dequant_kernel<T, MX_FP4_E8M0_32, false>);
        return launch_ex(k, dim3(unsigned(blocks)), dim3(kThreads), 0, 1, true, s, a);
    });
}

cudaError_t launch_fp4_gscale(const mx_fp4_layout& L, const void* X, mx_dtype dt, int64_t ldx, int64_t gsx,
                              float* gscale, cudaStream_t s) {
    cudaError_t e = cudaMemsetAsync(gscale, 0, size_t(L.groups) * 4, s);
    if (e != cudaSuccess) return e;
    if (L.rows > 0) {
        with_dtype(dt, [&](auto* tp) {
            using T = std::remove_pointer_t<decltype(tp)>;
            for (int g0 = 0; g0 < L.groups; g0 += 65535) {     // grid.y limit
                const int ng = L.groups - g0 < 65535 ? L.groups - g0 : 65535;
                const int bx = (L.rows + kWarps - 1) / kWarps;
                fp4_amax_kernel<T><<<dim3(bx < 1184 ? bx : 1184, ng), kThreads, 0, s>>>(
                    static_cast<const T*>(X) + int64_t(g0) * gsx, ldx, gsx, L.rows, L.K,
                    reinterpret_cast<uint32_t*>(gscale) + g0);
            }
            return 0;
        });
    }
    fp4_gscale_kernel<<<(L.groups + 255) / 256, 256, 0, s>>>(gscale, L.groups);
    return cudaGetLastError();
}

}  // namespace mx
