// experts.cu -- the routing around a layer of experts: slots sorted by expert,
// token rows gathered in that order, expert outputs summed back with the routing
// weights, and the gradients.
//
// Sort: a stable counting sort in one launch of one cluster.  Every warp owns a
// run of consecutive slots and counts them per expert in its own shared-memory row;
// the rows are scanned over the warps of a CTA, then over the CTAs (each CTA writes
// its totals into all of them), then over the experts; a second walk over the same
// slots writes each one's place, in the order of the lanes inside a group of 32.
// Lanes with the same expert are found from one ballot per bit of the expert: match.any
// takes time for each distinct value (8192 x 8 slots over 128 experts: 23 us with it).
//
// The row kernels move rows once: an item is one token (or slot) and a run of
// columns, held by one warp with its loads in flight together.  All are bound by
// HBM; a token's row is read once for all its slots.
#include <mutex>

#include "fp4.cuh"

namespace mx {
namespace {

using namespace fp4;

constexpr int kSortWarps = 32;
constexpr int kSortMaxCluster = 16;           // above the portable 8

struct SortArgs {
    const int32_t* ids;
    PlanPtrs p;
    int n, E;
    int chunk;        // slots per warp, a multiple of 32
    int bits;         // of the largest value, E
};

__device__ __forceinline__ uint32_t cl_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cl_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cl_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cl_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// a word of cluster CTA `rank` at the place of `p` in this one
__device__ __forceinline__ void st_remote(int* p, uint32_t rank, int v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(a) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// the lanes that hold the same value as this one, of values below 2^bits
__device__ __forceinline__ uint32_t same_lanes(int v, int bits) {
    uint32_t m = 0xffffffffu;
    for (int b = 0; b < bits; ++b) {
        const bool on = (v >> b) & 1;
        const uint32_t w = __ballot_sync(0xffffffffu, on);
        m &= on ? w : ~w;
    }
    return m;
}

// Every slot's expert of kBatch groups of 32, loaded together; E for a dropped or missing one.
constexpr int kBatch = 8;
__device__ __forceinline__ void load_ids(const SortArgs& a, int64_t s, int64_t s1, int (&ids)[kBatch]) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) ids[i] = s + 32 * i < s1 ? __ldg(a.ids + s + 32 * i) : -1;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) ids[i] = int(min(uint32_t(ids[i]), uint32_t(a.E)));
}

// dynamic shared memory: [warps][E] counts, [cluster][E] totals of every CTA, then [E] each:
// rows of the expert in the CTAs before this one, first row, first tile (and one word)
__global__ void __launch_bounds__(kSortWarps * 32) experts_sort_kernel(const __grid_constant__ SortArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    cl_arrive();                                              // waited for before the first remote write
    extern __shared__ int sm[];
    const int W = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = a.E, nc = int(cl_size());
    const uint32_t rank = cl_rank();
    int* const hist = sm;
    int* const totals = sm + W * E;
    int* const base = totals + nc * E;
    int* const first = base + E;
    int* const tile = first + E;
    int* const h = hist + warp * E;
    for (int i = threadIdx.x; i < W * E; i += blockDim.x) hist[i] = 0;
    __syncthreads();

    const int64_t s0 = (int64_t(rank) * W + warp) * a.chunk;
    const int64_t s1 = min(s0 + a.chunk, int64_t(a.n));
    int ids[kBatch];
    for (int64_t b = s0; b < s1; b += 32 * kBatch) {
        load_ids(a, b + lane, s1, ids);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (b + 32 * i >= s1) break;
            if (ids[i] < E) atomicAdd(h + ids[i], 1);
        }
    }
    __syncthreads();
    cl_wait();                                                // every CTA of the cluster runs
    for (int e = threadIdx.x; e < E; e += blockDim.x) {       // counts -> places within the CTA
        int run = 0;
#pragma unroll 8
        for (int w = 0; w < W; ++w) {
            const int c = hist[w * E + e];
            hist[w * E + e] = run;
            run += c;
        }
        for (int c = 0; c < nc; ++c) st_remote(totals + int(rank) * E + e, uint32_t(c), run);
    }
    cl_arrive();
    cl_wait();                                                // every CTA's totals are in place
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int before = 0, total = 0;
        for (int c = 0; c < nc; ++c) {
            const int t = totals[c * E + e];
            if (c < int(rank)) before += t;
            total += t;
        }
        base[e] = before;
        first[e] = total;
    }
    __syncthreads();
    if (warp == 0) {                                          // exclusive scans over the experts
        int rows = 0, tiles = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < E ? first[e] : 0, t = (c + kRows - 1) / kRows;
            int cs = c, ts = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, cs, o), v = __shfl_up_sync(0xffffffffu, ts, o);
                if (lane >= o) {
                    cs += u;
                    ts += v;
                }
            }
            if (e < E) {
                first[e] = rows + cs - c;
                tile[e] = tiles + ts - t;
                if (rank == 0) {
                    a.p.offsets[e] = rows + cs - c;
                    a.p.tiles[e] = tiles + ts - t;
                }
            }
            rows += __shfl_sync(0xffffffffu, cs, 31);
            tiles += __shfl_sync(0xffffffffu, ts, 31);
        }
        if (lane == 0) {
            tile[E] = rows;                                   // one word past: the number of kept rows
            if (rank == 0) {
                a.p.offsets[E] = rows;
                a.p.tiles[E] = tiles;
            }
        }
    }
    __syncthreads();
    for (int64_t b = s0; b < s1; b += 32 * kBatch) {
        if (s1 - s0 > 32 * kBatch) load_ids(a, b + lane, s1, ids);     // else still held
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (b + 32 * i >= s1) break;
            const int64_t s = b + 32 * i + lane;
            const int id = ids[i];
            const uint32_t same = same_lanes(id, a.bits);
            const int before = __popc(same & ((1u << lane) - 1));
            int at = 0;
            if (id < E) at = h[id];
            __syncwarp();
            if (id < E && before == 0) h[id] = at + __popc(same);
            __syncwarp();
            if (id < E) {
                const int in_e = base[id] + at + before, p = first[id] + in_e;
                a.p.order[p] = int(s);                        // the only store that scatters
                a.p.pos[s] = p;
                a.p.dest[s] = tile[id] * kRows + in_e;
            } else if (s < s1) {
                a.p.pos[s] = -1;
                a.p.dest[s] = -1;
            }
        }
    }
    for (int64_t p = int64_t(tile[E]) + rank * blockDim.x + threadIdx.x; p < a.n; p += int64_t(nc) * blockDim.x)
        a.p.order[p] = -1;
}

// ---------------------------------------------------------------- row kernels
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// A chunk of EL elements as it lies in memory: eight with 16-byte accesses, or one.  Loads are
// kept in this form, which takes half the registers of fp32 values, until they are used.
template <int EL, typename T> struct Chunk {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < int(sizeof(T) / 2); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < int(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
    }
    __device__ __forceinline__ void values(float (&v)[EL]) const { load8v(reinterpret_cast<const T*>(w), v); }
};
template <typename T> struct Chunk<1, T> {
    T w;
    __device__ __forceinline__ void load(const T* p) { w = *p; }
    __device__ __forceinline__ void store(T* p) const { *p = w; }
    __device__ __forceinline__ void values(float (&v)[1]) const { v[0] = to_f32(w); }
};
template <int EL, typename T> __device__ __forceinline__ void store_chunk(T* p, const float (&v)[EL]) {
    if constexpr (EL == 8) store8v(p, v);
    else *p = from_f32<T>(v[0]);
}

// Rows are split into runs of NI * 32 chunks.  With eight-element chunks the columns past the
// last whole chunk are taken one by one by the lanes of the row's last run.
template <int EL, int NI> int runs_of(int H) { return (H + NI * 32 * EL - 1) / (NI * 32 * EL); }

// for the whole chunks i (first column c) of run `run` that this lane holds
#define MX_FOR_CHUNKS(i, c, NI, run, H)                   \
    _Pragma("unroll") for (int i = 0; i < NI; ++i)        \
        if (const int c = (run) * (NI * 32 * EL) + (i * 32 + lane) * EL; c + EL <= (H))

constexpr int kGatherIter = 4, kCombineIter = 2, kCombineRows = 4, kBwdIter = 4;

// copies X[t] to the rows of the token's kept slots
template <typename T, int EL>
__global__ void __launch_bounds__(kThreads)
gather_kernel(const int32_t* pos, int T_, int k, int H, int runs, const T* X, int64_t ldx, T* Xs, int64_t lds) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int NI = kGatherIter;
    const int lane = threadIdx.x & 31;
    const unsigned item = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t t = item / unsigned(runs);
    const int run = int(item % unsigned(runs));
    if (t >= T_) return;
    const T* x = X + t * ldx;
    const int32_t* ps = pos + t * k;
    const int tail = EL > 1 ? H / EL * EL + lane : H;      // this lane's tail column
    const bool has_tail = EL > 1 && run == runs - 1 && tail < H;
    Chunk<EL, T> v[NI];
    MX_FOR_CHUNKS(i, c, NI, run, H) v[i].load(x + c);
    T vt{};
    if (has_tail) vt = x[tail];
#pragma unroll 4
    for (int j = 0; j < k; ++j) {
        const int p = ps[j];
        if (p < 0) continue;
        T* o = Xs + int64_t(p) * lds;
        MX_FOR_CHUNKS(i, c, NI, run, H) v[i].store(o + c);
        if (has_tail) o[tail] = vt;
    }
}

// Y[t] = sum_j w[t, j] Ys[pos[t, j]] in fp32, in slot order, rounded once; w NULL: plain sum.
// kCombineRows rows are in flight together.
template <typename S, typename T, int EL>
__global__ void __launch_bounds__(kThreads)
combine_kernel(const int32_t* pos, const float* w, int T_, int k, int H, int runs, const S* Ys, int64_t lds, T* Y,
               int64_t ldy) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int NI = kCombineIter;
    const int lane = threadIdx.x & 31;
    const unsigned item = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t t = item / unsigned(runs);
    const int run = int(item % unsigned(runs));
    if (t >= T_) return;
    const int tail = EL > 1 ? H / EL * EL + lane : H;
    const bool has_tail = EL > 1 && run == runs - 1 && tail < H;
    float acc[NI][EL], at = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < EL; ++e) acc[i][e] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += kCombineRows) {
        int p[kCombineRows];
        float wj[kCombineRows];
#pragma unroll
        for (int j = 0; j < kCombineRows; ++j) {
            const bool in = j0 + j < k;
            p[j] = in ? pos[t * k + j0 + j] : -1;
            wj[j] = in && w ? w[t * k + j0 + j] : 1.0f;
        }
        Chunk<EL, S> v[kCombineRows][NI];
        float vt[kCombineRows];
#pragma unroll
        for (int j = 0; j < kCombineRows; ++j) {
            if (p[j] < 0) continue;
            const S* y = Ys + int64_t(p[j]) * lds;
            MX_FOR_CHUNKS(i, c, NI, run, H) v[j][i].load(y + c);
            vt[j] = has_tail ? to_f32(y[tail]) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < kCombineRows; ++j) {
            if (p[j] < 0) continue;
            MX_FOR_CHUNKS(i, c, NI, run, H) {
                float f[EL];
                v[j][i].values(f);
#pragma unroll
                for (int e = 0; e < EL; ++e) acc[i][e] = __fmaf_rn(wj[j], f[e], acc[i][e]);
            }
            at = __fmaf_rn(wj[j], vt[j], at);
        }
    }
    T* o = Y + t * ldy;
    MX_FOR_CHUNKS(i, c, NI, run, H) store_chunk<EL>(o + c, acc[i]);
    if (has_tail) o[tail] = from_f32<T>(at);
}

// One warp per slot: dYs row = w * dY row, dw = <dY row, Ys row>.  The warps of a token's
// slots are neighbours, so its dY row is read from HBM once.
template <typename T, int EL>
__global__ void __launch_bounds__(kThreads)
combine_bwd_kernel(const int32_t* pos, const float* w, int64_t n, int k, int H, int runs, const T* dY, int64_t ldy,
                   const T* Ys, int64_t lds, T* dYs, int64_t ldds, float* dw) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int NI = kBwdIter;
    const int lane = threadIdx.x & 31;
    const int64_t s = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (s >= n) return;
    const int p = pos[s];
    if (p < 0) {
        if (lane == 0) dw[s] = 0.0f;
        return;
    }
    const float ws = w[s];
    const T* g = dY + (s / k) * ldy;
    const T* y = Ys + int64_t(p) * lds;
    T* o = dYs + int64_t(p) * ldds;
    float dot = 0.0f;
    for (int run = 0; run < runs; ++run) {
        Chunk<EL, T> a[NI], b[NI];
        MX_FOR_CHUNKS(i, c, NI, run, H) {
            a[i].load(g + c);
            b[i].load(y + c);
        }
        MX_FOR_CHUNKS(i, c, NI, run, H) {
            float u[EL], v[EL];
            a[i].values(u);
            b[i].values(v);
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                dot = __fmaf_rn(u[e], v[e], dot);
                u[e] = __fmul_rn(u[e], ws);
            }
            store_chunk<EL>(o + c, u);
        }
    }
    if (const int c = EL > 1 ? H / EL * EL + lane : H; c < H) {
        const float a = to_f32(g[c]);
        dot = __fmaf_rn(a, to_f32(y[c]), dot);
        o[c] = from_f32<T>(__fmul_rn(a, ws));
    }
#pragma unroll
    for (int o2 = 16; o2 > 0; o2 >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o2);
    if (lane == 0) dw[s] = dot;
}

bool vec_ok(const void* p, int64_t ld, int esz) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * esz) % 16 == 0;
}

// once per device: what the sort's kernel may take, and whether a cluster of its largest size with the most
// shared memory can be placed (16 free SMs side by side)
cudaError_t sort_prepare(bool* wide) {
    static struct { bool done, wide; } known[64];
    static std::mutex lock;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> hold(lock);
    if (!known[dev].done) {
        constexpr int kSmem = ((kSortWarps + kSortMaxCluster + 3) * kMaxExperts + 1) * 4;
        e = cudaFuncSetAttribute(experts_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(experts_sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kSortMaxCluster);
        cfg.blockDim = dim3(kSortWarps * 32);
        cfg.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = kSortMaxCluster;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, experts_sort_kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        known[dev] = {true, n > 0};
    }
    *wide = known[dev].wide;
    return cudaSuccess;
}

cudaError_t blocks_of(int64_t items, unsigned* blocks) {
    if (items > 0xFFFFFF00ll) return cudaErrorInvalidConfiguration;      // items are counted in 32 bits
    *blocks = unsigned((items + kWarps - 1) / kWarps);
    return cudaSuccess;
}

}  // namespace

// CTAs of the sort's cluster.  1024 slots are one group of 32 for each warp of one CTA.  The stores of
// `order` scatter, and a CTA writes about a sector a cycle, so many slots go to 16 CTAs (65536 over 128
// experts: 8.4 us, 10.9 with 8) where the device can place a cluster of that size, which is above the portable 8.
int sort_ctas(int n, bool wide) {
    return n > 16384 && wide ? kSortMaxCluster : n > 4096 ? 8 : n > 2048 ? 4 : n > 1024 ? 2 : 1;
}

cudaError_t launch_experts_sort_on(const mx_experts_layout& P, const int32_t* ids, void* plan, int ctas, cudaStream_t s) {
    int warps = (P.n + 31) / 32;
    warps = warps < 1 ? 1 : warps > kSortWarps ? kSortWarps : warps;
    SortArgs a{};
    a.ids = ids;
    a.p = plan_ptrs(P, plan);
    a.n = P.n;
    a.E = P.E;
    const int64_t per = (int64_t(P.n) + int64_t(ctas) * warps - 1) / (int64_t(ctas) * warps);
    a.chunk = int((per + 31) / 32 * 32);
    a.bits = 32 - __builtin_clz(unsigned(P.E));
    const size_t smem = (size_t(warps + ctas + 3) * P.E + 1) * sizeof(int);
    return launch_ex(experts_sort_kernel, dim3(ctas), dim3(warps * 32), smem, ctas, true, s, a);
}

cudaError_t launch_experts_sort(const mx_experts_layout& P, const int32_t* ids, void* plan, cudaStream_t s) {
    bool wide = false;
    if (const cudaError_t e = sort_prepare(&wide); e != cudaSuccess) return e;
    return launch_experts_sort_on(P, ids, plan, sort_ctas(P.n, wide), s);
}

cudaError_t launch_experts_gather(const mx_experts_layout& P, const void* plan, const void* X, mx_dtype dt, int H,
                                  int64_t ldx, void* Xs, int64_t lds, cudaStream_t s) {
    const int esz = dtype_bytes(dt);
    const bool vec = vec_ok(X, ldx, esz) && vec_ok(Xs, lds, esz);
    const int32_t* pos = plan_ptrs(P, plan).pos;
    return with_dtype(dt, [&](auto* tp) {
        using T = std::remove_pointer_t<decltype(tp)>;
        const int runs = vec ? runs_of<8, kGatherIter>(H) : runs_of<1, kGatherIter>(H);
        unsigned nb;
        cudaError_t e = blocks_of(int64_t(P.T) * runs, &nb);
        if (e != cudaSuccess) return e;
        auto k = vec ? gather_kernel<T, 8> : gather_kernel<T, 1>;
        return launch_ex(k, dim3(nb), dim3(kThreads), 0, 1, true, s, pos, P.T, P.k, H, runs, static_cast<const T*>(X),
                         ldx, static_cast<T*>(Xs), lds);
    });
}

cudaError_t launch_experts_combine(const mx_experts_layout& P, const void* plan, const void* Ys, mx_dtype sdt, int H,
                                   int64_t lds, const float* w, void* Y, mx_dtype ydt, int64_t ldy, cudaStream_t s) {
    const bool vec = vec_ok(Ys, lds, dtype_bytes(sdt)) && vec_ok(Y, ldy, dtype_bytes(ydt));
    const int32_t* pos = plan_ptrs(P, plan).pos;
    return with_dtype(sdt, [&](auto* sp) {
        using S = std::remove_pointer_t<decltype(sp)>;
        return with_dtype(ydt, [&](auto* tp) {
            using T = std::remove_pointer_t<decltype(tp)>;
            const int runs = vec ? runs_of<8, kCombineIter>(H) : runs_of<1, kCombineIter>(H);
            unsigned nb;
            cudaError_t e = blocks_of(int64_t(P.T) * runs, &nb);
            if (e != cudaSuccess) return e;
            auto k = vec ? combine_kernel<S, T, 8> : combine_kernel<S, T, 1>;
            return launch_ex(k, dim3(nb), dim3(kThreads), 0, 1, true, s, pos, w, P.T, P.k, H, runs,
                             static_cast<const S*>(Ys), lds, static_cast<T*>(Y), ldy);
        });
    });
}

cudaError_t launch_experts_combine_bwd(const mx_experts_layout& P, const void* plan, const void* dY, const void* Ys,
                                       mx_dtype dt, int H, int64_t ldy, int64_t lds, const float* w, void* dYs,
                                       int64_t ldds, float* dw, cudaStream_t s) {
    const int esz = dtype_bytes(dt);
    const bool vec = vec_ok(dY, ldy, esz) && vec_ok(Ys, lds, esz) && vec_ok(dYs, ldds, esz);
    const int32_t* pos = plan_ptrs(P, plan).pos;
    return with_dtype(dt, [&](auto* tp) {
        using T = std::remove_pointer_t<decltype(tp)>;
        const int runs = vec ? runs_of<8, kBwdIter>(H) : runs_of<1, kBwdIter>(H);
        unsigned nb;
        cudaError_t e = blocks_of(P.n, &nb);
        if (e != cudaSuccess) return e;
        auto k = vec ? combine_bwd_kernel<T, 8> : combine_bwd_kernel<T, 1>;
        return launch_ex(k, dim3(nb), dim3(kThreads), 0, 1, true, s, pos, w, int64_t(P.n), P.k, H, runs,
                         static_cast<const T*>(dY), ldy, static_cast<const T*>(Ys), lds, static_cast<T*>(dYs), ldds, dw);
    });
}

}  // namespace mx
