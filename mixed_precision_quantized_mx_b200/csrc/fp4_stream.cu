// fp4_stream.cu -- the FP4 product for few tokens: one CTA per 128 weight rows and up to 128
// tokens, bound by the weights' bytes.
//
// A ring of stages (one k-block of weights, 17 or 18 KB in one bulk copy, and its tokens) keeps
// the copies ahead across tiles.  The MMA's N follows the tokens that are there: one token costs
// N = 8 columns.  With few row tiles a cluster of CTAs shares a tile's K range and adds the partial
// sums in CTA order.  Up to 4 tokens each CTA sends column c to CTA c mod S by st.async (data and
// completion in one, so no fence), about 0.25 us a column.  With more it leaves its sums in its own
// shared memory and each CTA reads a share of the columns from all of them, 16 bytes a lane: about 2.5
// us and 0.012 a column (1024 x 8192, 16 tokens: 8.2 us sent, 7.6 read; 4096 x 14336, 64 tokens: 16.9
// us by one CTA, 13.4 by four).
//
// Up to 4 tokens the kernel quantises them itself: every CTA reads the token rows of its K
// range (they stay in L2) and eight warps write codes and scales straight into the stages,
// laid out as stored activations are, so the call is one launch and the weights stream from its
// start.  (With more tokens the work repeated in every CTA costs more than the quantiser's launch:
// 28672 x 8192 at 5 tokens 30.6 us against 25.0.)  An MMA's scales have to start at a TMEM column
// that is a multiple of four, so the scales of several steps cannot share one copy.
//
// Roles: warp 0 weight copies, 1-2 MMAs (and TMEM), 3 token copies, 4-7 epilogue (a warp per TMEM
// lane quarter), 8-15 quantisers.  Single lanes copy: a turn (wait, arm, one copy) measured 118 ns and
// each further copy of the same lane 24 ns, copies spread over lanes 50 ns more each.  An MMA warp
// waits once and commits once per stage and issues from converged code; its turn takes about
// 350 ns, which is more than a CTA's share of HBM needs, so two warps take alternate stages
// (28672 x 8192, one token: 28.0 us with one, 22.3 with two, 20.5 at the measured copy rate).
// Scales in TMEM have a buffer per stage, free when the stage has been filled again.
#include "fp4_mma.cuh"
#include "fp4_quant.cuh"

namespace mx {
namespace fp4 {
namespace {

// NT: most tokens of a unit (16, 64 or 128; below 128 all tokens of an expert, as a unit's tokens
// start at a stored tile); SPLIT: the cluster shares a unit's K range; FUSED: tokens quantised here
template <int FMT, int NT, bool SPLIT, bool FUSED> struct StreamCfg {
    static_assert(NT == 16 || !FUSED, "only few tokens are quantised here");
    static constexpr bool kPull = SPLIT && !FUSED;        // how the CTAs exchange partial sums
    static constexpr int kScale = scale_bytes<FMT>();
    static constexpr int kW = tile_bytes<FMT>();
    static constexpr int kT = NT * 128 + kScale;
    static constexpr int kStages = NT == 16 ? 8 : NT == 128 && SPLIT ? 4 : 6;   // as shared memory has room for
    static constexpr int kRed = SPLIT ? NT * kRows : 1;   // floats of one buffer of the exchange
    static constexpr int kSfCols = kScale / 512 * 4;      // TMEM columns of one operand's scales
    // MMA warps, which take alternate stages into accumulators of their own.  A place of the ring
    // has to belong to one of them: each waits on every phase of the barriers that it waits on.
    static constexpr int kIssuers = 2;
    static_assert(kStages % kIssuers == 0, "a place of the ring belongs to one issuer");
    // units whose accumulators fit beside every stage's scales
    static constexpr int kSlots = NT == 128 ? 1 : 2;
    static constexpr int kSlot = kIssuers * NT;           // columns of a unit's accumulators
    static constexpr int kSf0 = kSlots * kSlot;
    static constexpr int kTmem = 512;
    static_assert(kSf0 + kStages * 2 * kSfCols <= kTmem, "accumulators and scales fit in TMEM");
    static_assert(kW % 1024 == 0 && kT % 1024 == 0, "operands start at the swizzle's period");
    struct __align__(1024) Smem {
        uint8_t W[kStages][kW];
        uint8_t T[kStages][kT];
        float red[kPull ? 1 : 2][kRed];  // [column][row], or [buffer][source CTA][own column][row]
        ExpertTable table;
        uint64_t full[kStages];          // weights and tokens are in place (an arrival each)
        uint64_t empty[kStages];         // the MMAs that read the stage completed
        uint64_t acc_full[2], acc_empty[2];
        uint64_t red_full[2], red_free[2];   // partial sums of every CTA in place / read by every CTA
        uint64_t mma_done[2];
        uint32_t tmem_base;
        int abort;
    };
};

constexpr int kQuantWarps = 8;
constexpr int kCopyThreads = 256, kFusedThreads = kCopyThreads + 32 * kQuantWarps;

// COLS columns of a unit's sums: the issuers' accumulators (NT columns apart) added.  A unit of one
// stage has only the one of that stage's issuer.
template <int NT, int COLS>
__device__ __forceinline__ void sums(uint32_t addr, int stages, int first_stage, float (&v)[COLS]) {
    uint32_t r[COLS], r2[COLS];
    tmem_cols<COLS>(addr, r);
    tmem_cols<COLS>(addr + NT, r2);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
        const float x = __uint_as_float(r[c]), y = __uint_as_float(r2[c]);
        v[c] = stages > 1 ? x + y : (first_stage & 1) ? y : x;
    }
}

// XT: the tokens' type when the kernel quantises them, else void
template <int FMT, int NT, bool SPLIT, typename XT>
__global__ void __launch_bounds__(std::is_void_v<XT> ? kCopyThreads : kFusedThreads, 1)
fp4_stream_kernel(const __grid_constant__ GemmArgs a) {
    constexpr bool FUSED = !std::is_void_v<XT>;
    using C = StreamCfg<FMT, NT, SPLIT, FUSED>;
    extern __shared__ uint8_t smem_raw[];
    typename C::Smem& S =
        *reinterpret_cast<typename C::Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank = 0, nc = 1;
    if constexpr (SPLIT) {
        rank = cluster_ctarank();
        asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(nc));
    }
    const int cid = int(blockIdx.x / nc), ncl = int(gridDim.x / nc);
    const int kb0 = int(int64_t(a.nkb) * rank / nc), kb1 = int(int64_t(a.nkb) * (rank + 1) / nc);
    volatile int* abort = &S.abort;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&S.full[s], 2);
            mbar_init(&S.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&S.acc_full[b], C::kIssuers);
            mbar_init(&S.acc_empty[b], 4);
            mbar_init(&S.red_full[b], C::kPull ? 4 * nc : 1);
            mbar_init(&S.red_free[b], 4 * nc);
        }
        for (int b = 0; b < 2; ++b) mbar_init(&S.mma_done[b], 1);
        S.abort = 0;
        fence_mbar_init();
    }
    if (warp == 2) {
        tmem_alloc(&S.tmem_base, C::kTmem);
        tmem_relinquish();
    }
    // With `early` the kernel before this one is the quantiser of its tokens, which lets this one
    // launch only after its own wait: the weights and the plan are complete, the tokens are not.
    if (!a.early) grid_wait();
    if (a.E > 0) {
        for (int i = threadIdx.x; i <= a.E; i += blockDim.x) {
            S.table.offsets[i] = a.offsets[i];
            S.table.tiles[i] = a.tiles[i];
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if constexpr (SPLIT) cluster_arrive();       // this CTA's barriers are initialised; the copies start
    const uint32_t tmem = S.tmem_base;
    Walk w{};
    walk_expert(w, a, S.table, NT);

    if (warp == 0) {
        // ---------------------------------------------------- weight tiles
        if (lane == 0) {
            int it = 0;
            for (int u = cid; !a.stall && walk_to(w, u, a.R, a, S.table, NT); u += ncl) {
                const uint8_t* src = a.W + ((uint64_t(w.e) * a.R + w.rt) * a.nkb + kb0) * C::kW;
                for (int kb = kb0; kb < kb1; ++kb, ++it, src += C::kW) {
                    const int s = it % C::kStages;
                    if (!mbar_wait_bounded(&S.empty[s], ((it / C::kStages) & 1) ^ 1, abort, a.status, a.timeout_ns))
                        goto weights_out;
                    mbar_arrive_expect_tx(&S.full[s], C::kW);
                    bulk_g2s(S.W[s], src, C::kW, &S.full[s]);
                }
            }
        weights_out:
            drain<C::kStages>(S.full, it, a.timeout_ns);
        }
    } else if (warp == 3) {
        // ---------------------------------------------------- stored tokens and their scales
        if (!FUSED && lane == 0) {
            int it = 0;
            grid_wait();
            for (int u = cid; !a.stall && walk_to(w, u, a.R, a, S.table, NT); u += ncl) {
                const uint8_t* src = a.A + (uint64_t(w.tile0 + w.tt) * a.nkb + kb0) * C::kW;
                const uint32_t bytes = uint32_t((w.ntok + 7) & ~7) * 128;
                for (int kb = kb0; kb < kb1; ++kb, ++it, src += C::kW) {
                    const int s = it % C::kStages;
                    if (!mbar_wait_bounded(&S.empty[s], ((it / C::kStages) & 1) ^ 1, abort, a.status, a.timeout_ns))
                        goto tokens_out;
                    mbar_arrive_expect_tx(&S.full[s], bytes + C::kScale);
                    bulk_g2s(S.T[s], src, bytes, &S.full[s]);
                    bulk_g2s(S.T[s] + NT * 128, src + kCodeBytes, C::kScale, &S.full[s]);
                }
            }
        tokens_out:
            drain<C::kStages>(S.full, it, a.timeout_ns);
        }
    } else if (warp == 1 || warp == 2) {
        // ---------------------------------------------------- MMAs
        const int mine = warp - 1;
        const uint64_t wd0 = sw128_kmajor_desc(smem_u32(S.W[0])), td0 = sw128_kmajor_desc(smem_u32(S.T[0]));
        const uint64_t wf0 = scale_desc(smem_u32(S.W[0]) + kCodeBytes), tf0 = scale_desc(smem_u32(S.T[0]) + NT * 128);
        int it0 = 0;                                 // first stage of the unit, of the CTA's
        uint32_t uc = 0;
        for (int u = cid; walk_to(w, u, a.R, a, S.table, NT); u += ncl, ++uc, it0 += kb1 - kb0) {
            const uint32_t slot = uc % C::kSlots;
            const uint32_t d = tmem + slot * C::kSlot + mine * NT;
            const int n = (w.ntok + 7) & ~7;
            bool ok = mbar_wait_bounded(&S.acc_empty[slot], ((uc / C::kSlots) & 1) ^ 1, abort, a.status, a.timeout_ns);
            if (!__all_sync(0xffffffffu, ok)) goto mma_out;
            const int first = kb0 + ((it0 ^ mine) & 1);    // of this warp's k-blocks
            for (int kb = first; kb < kb1; kb += C::kIssuers) {
                const int it = it0 + kb - kb0, s = it % C::kStages;
                ok = mbar_wait_bounded(&S.full[s], (it / C::kStages) & 1, abort, a.status, a.timeout_ns);
                if (!__all_sync(0xffffffffu, ok)) goto mma_out;
                tc_fence_after();
                const uint32_t sfa = tmem + C::kSf0 + s * 2 * C::kSfCols, sfb = sfa + C::kSfCols;
                // addresses are below 2^18, so descriptors of later stages and steps are sums
                const uint64_t wo = uint64_t(s * (C::kW / 16)), to = uint64_t(s * (C::kT / 16));
                const int steps = kb == a.nkb - 1 ? a.last_steps : kSteps;
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < C::kScale / 512; ++j) {
                        copy_scales<1>(sfa + 4 * j, wf0 + wo + 32 * j);
                        copy_scales<1>(sfb + 4 * j, tf0 + to + 32 * j);
                    }
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        const uint32_t word = FMT == MX_FP4_E4M3_16 ? k : k >> 1;
                        const uint32_t sfid = FMT == MX_FP4_E4M3_16 ? 0 : 2 * (k & 1);
                        if (k < steps)
                            mma_fp4<FMT, 1>(d, wd0 + wo + 2 * k, td0 + to + 2 * k, idesc_fp4<FMT>(kRows, n, sfid),
                                            sfa + 4 * word, sfb + 4 * word, kb > first || k > 0 ? 1u : 0u);
                    }
                    mma_commit(&S.empty[s]);
                }
                __syncwarp();
            }
            if (elect_one()) mma_commit(&S.acc_full[slot]);
            __syncwarp();
        }
    mma_out:
        if (elect_one()) mma_commit(&S.mma_done[mine]);    // every MMA has completed before the teardown
        __syncwarp();
        int dummy = 0;
        mbar_wait_bounded(&S.mma_done[mine], 0, &dummy, nullptr, a.timeout_ns);
    } else if (warp >= 4 && warp < 8) {
        // ---------------------------------------------------- epilogue
        const int q = warp & 3, row = q * 32 + lane, nk = kb1 - kb0;
        if constexpr (SPLIT) cluster_wait();     // every CTA's are
        grid_wait();
        grid_launch();                           // after the wait: what a dependent may read early is complete
        const float ga = FUSED ? (a.gscale ? *a.gscale : 1.0f) : *a.ga;
        uint32_t uc = 0;
        for (int u = cid; walk_to(w, u, a.R, a, S.table, NT); u += ncl, ++uc) {
            const uint32_t slot = uc % C::kSlots;
            const int nf = w.rt * kRows + row;   // output feature
            const int64_t row0 = int64_t(w.row0) + int64_t(w.tt) * NT;
            const OutScale scale = out_scale(ga, a.gw[w.e]);
            bool ok = mbar_wait_bounded(&S.acc_full[slot], (uc / C::kSlots) & 1, abort, a.status, a.timeout_ns);
            if (!__all_sync(0xffffffffu, ok)) goto epi_done;
            tc_fence_after();
            const uint32_t d = tmem + (uint32_t(q * 32) << 16) + slot * C::kSlot;
            if constexpr (!SPLIT) {
                // all columns to registers, then the accumulators are free for the next unit's MMAs while
                // these are stored
                constexpr int CC = NT == 16 ? 8 : 16;
                float v[NT / CC][CC];
#pragma unroll
                for (int j = 0; j < NT / CC; ++j)
                    if (j * CC < w.ntok) sums<NT, CC>(d + j * CC, nk, int(uc) * nk, v[j]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.acc_empty[slot]);
#pragma unroll
                for (int j = 0; j < NT / CC; ++j) {
                    if (j * CC < w.ntok) {
#pragma unroll
                        for (int c = 0; c < CC; ++c) v[j][c] = scaled(v[j][c], scale);
                        store_cols<CC>(a, row0 + j * CC, w.ntok - j * CC, nf, v[j]);
                    }
                }
            } else if constexpr (C::kPull) {
                // this CTA's partial sums to its own shared memory, then a share of the columns from
                // all CTAs': a warp reads whole columns, every fourth of the share
                float* const red = S.red[0];
                if (uc > 0) {
                    ok = wait_cluster(&S.red_free[0], (uc - 1) & 1, abort, a.status, a.timeout_ns);
                    if (!__all_sync(0xffffffffu, ok)) goto epi_done;
                }
#pragma unroll
                for (int c0 = 0; c0 < NT; c0 += 16) {
                    if (c0 < w.ntok) {
                        float v[16];
                        sums<NT, 16>(d + c0, nk, int(uc) * nk, v);
#pragma unroll
                        for (int c = 0; c < 16; ++c) red[(c0 + c) * kRows + row] = v[c];
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.acc_empty[slot]);
                if (lane < nc) arrive_release_cluster(mapa_shared(&S.red_full[0], lane));
                ok = wait_cluster(&S.red_full[0], uc & 1, abort, a.status, a.timeout_ns);
                if (!__all_sync(0xffffffffu, ok)) goto epi_done;
                const int per = (w.ntok + int(nc) - 1) / int(nc), c1 = min(w.ntok, (int(rank) + 1) * per);
                for (int c0 = int(rank) * per + q; c0 < c1; c0 += 16) {   // columns c0, c0 + 4, ..
                    float v[4][4] = {};
                    for (uint32_t s0 = 0; s0 < nc; s0 += 4) {             // added in CTA order
                        float4 x[4][4];
#pragma unroll
                        for (uint32_t s = 0; s < 4; ++s) {
                            if (s0 + s < nc) {
                                const uint32_t from = mapa_shared(&red[c0 * kRows + 4 * lane], s0 + s);
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    if (c0 + 4 * c < c1) x[s][c] = ld_cluster(from + 4 * c * kRows * 4);
                            }
                        }
#pragma unroll
                        for (uint32_t s = 0; s < 4; ++s) {
                            if (s0 + s < nc) {
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    if (c0 + 4 * c < c1) {
                                        v[c][0] += x[s][c].x;
                                        v[c][1] += x[s][c].y;
                                        v[c][2] += x[s][c].z;
                                        v[c][3] += x[s][c].w;
                                    }
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (c0 + 4 * c < c1) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[c][i] = scaled(v[c][i], scale);
                            store_four(a, row0 + c0 + 4 * c, w.rt * kRows + 4 * lane, v[c]);
                        }
                    }
                }
                __syncwarp();
                if (lane < nc) arrive_release_cluster(mapa_shared(&S.red_free[0], lane));
            } else {
                // this CTA's partial sums to the CTAs that own the columns, then the own columns
                const uint32_t b = uc & 1, use = uc >> 1;
                if (use > 0) {
                    ok = wait_cluster(&S.red_free[b], (use - 1) & 1, abort, a.status, a.timeout_ns);
                    if (!__all_sync(0xffffffffu, ok)) goto epi_done;
                }
                const int per = (w.ntok + int(nc) - 1) / int(nc);                       // most columns of an owner
                const int own = (w.ntok - int(rank) + int(nc) - 1) / int(nc);           // this CTA's
                float* const red = S.red[b];
                if (q == 0 && lane == 0) mbar_arrive_expect_tx(&S.red_full[b], uint32_t(max(own, 0)) * nc * kRows * 4);
                for (int c0 = 0; c0 < w.ntok; c0 += 8) {
                    float v[8];
                    sums<NT, 8>(d + c0, nk, int(uc) * nk, v);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const int col = c0 + c;
                        if (col < w.ntok) {
                            const uint32_t to = uint32_t(col) % nc;
                            st_async(mapa_shared(&red[(int(rank) * per + col / int(nc)) * kRows + row], to),
                                     v[c], mapa_shared(&S.red_full[b], to));
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.acc_empty[slot]);
                ok = wait_cluster(&S.red_full[b], use & 1, abort, a.status, a.timeout_ns);
                if (!__all_sync(0xffffffffu, ok)) goto epi_done;
                for (int i = 0; i < own; ++i) {
                    float v[1] = {0.0f};
                    for (uint32_t c = 0; c < nc; ++c) v[0] += red[(int(c) * per + i) * kRows + row];
                    v[0] = scaled(v[0], scale);
                    store_cols<1>(a, row0 + int(rank) + i * int(nc), 1, nf, v);
                }
                __syncwarp();                    // the warp's reads come before other CTAs' next sums
                if (lane < nc) arrive_release_cluster(mapa_shared(&S.red_free[b], lane));
            }
        }
    epi_done:;
    } else if (warp >= 8) {
        // ---------------------------------------------------- quantisers
        // The warps take stages in turn: eight lanes a token row, 32 columns a lane.  Each loads its
        // next stage's columns while it quantises one and waits for its place.
        if constexpr (FUSED) {
            // a place of the ring belongs to one warp, which so waits on every phase of its barrier
            static_assert(C::kStages % kQuantWarps == 0, "a place of the ring belongs to one quantiser");
            grid_wait();
            const MatrixScale m = matrix_scale(a.gscale ? *a.gscale : 1.0f);
            const int r = lane >> 3, ch = lane & 7, nk = kb1 - kb0;
            int u = cid, it0 = 0;                        // the unit that holds a stage, its first stage
            bool live = false;                           // the lane has a row of it
            Columns<XT> cur, next;
            auto fetch = [&](Columns<XT>& c, int it) {   // false past the last stage
                while (it >= it0 + nk) {
                    u += ncl;
                    it0 += nk;
                }
                if (a.stall || !walk_to(w, u, a.R, a, S.table, NT)) return false;
                live = r < w.ntok;
                if (live) {
                    int64_t at = int64_t(w.row0) + int64_t(w.tt) * NT + r;
                    if (a.order) at = a.order[at] / a.k;
                    const XT* const x = static_cast<const XT*>(a.X) + at * a.ldx;
                    const int c0 = (kb0 + it - it0) * kCols + ch * 32;
                    if (a.aligned) c.template load<true>(x, c0, a.K);
                    else c.template load<false>(x, c0, a.K);
                }
                return true;
            };
            int it = warp - 8;
            bool more = fetch(cur, it);
            while (more) {
                const bool now = live;
                more = fetch(next, it + kQuantWarps);
                uint32_t codes[4], sb = 0;
                if (now) sb = quant_columns<FMT>(cur, m, codes);
                const int s = it % C::kStages;
                const bool ok = mbar_wait_bounded(&S.empty[s], ((it / C::kStages) & 1) ^ 1, abort, a.status, a.timeout_ns);
                if (!__all_sync(0xffffffffu, ok)) break;
                if (now) {
                    uint8_t* const t = S.T[s];
                    uint8_t* const f = t + NT * 128 + 16 * r;
                    *reinterpret_cast<uint4*>(t + r * 128 + ((ch ^ r) << 4)) =
                        make_uint4(codes[0], codes[1], codes[2], codes[3]);
                    if constexpr (FMT == MX_FP4_E4M3_16)
                        *reinterpret_cast<uint16_t*>(f + 512 * (ch >> 1) + 2 * (ch & 1)) = uint16_t(sb);
                    else
                        f[512 * (ch >> 2) + (ch & 3)] = uint8_t(sb);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.full[s]);
                cur = next;
                it += kQuantWarps;
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    if constexpr (SPLIT) {
        if (warp < 4 || warp >= 8) cluster_wait();
        cluster_sync();                          // no CTA's shared memory is used after it has left
    } else {
        __syncthreads();
    }
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmem);
    }
}

template <int FMT, int NT, bool SPLIT, bool FUSED> constexpr size_t stream_smem() {
    constexpr size_t bytes = sizeof(typename StreamCfg<FMT, NT, SPLIT, FUSED>::Smem) + 1024;
    static_assert(bytes <= 232448, "shared memory of a CTA");
    return bytes;
}

// f(kernel, dynamic shared memory, threads) for every instance / for the one that serves a call
template <int FMT, int NT, bool SPLIT, typename XT, typename F> cudaError_t with_kernel(F f) {
    constexpr bool FUSED = !std::is_void_v<XT>;
    return f(fp4_stream_kernel<FMT, NT, SPLIT, XT>, stream_smem<FMT, NT, SPLIT, FUSED>(),
             FUSED ? kFusedThreads : kCopyThreads);
}
template <int FMT, bool SPLIT, typename F> cudaError_t every_kernel(F f) {
    cudaError_t e = with_kernel<FMT, 16, SPLIT, void>(f);
    if (e == cudaSuccess) e = with_kernel<FMT, 16, SPLIT, float>(f);
    if (e == cudaSuccess) e = with_kernel<FMT, 16, SPLIT, __half>(f);
    if (e == cudaSuccess) e = with_kernel<FMT, 16, SPLIT, __nv_bfloat16>(f);
    if (e == cudaSuccess) e = with_kernel<FMT, 64, SPLIT, void>(f);
    if (e == cudaSuccess) e = with_kernel<FMT, 128, SPLIT, void>(f);
    return e;
}
template <int FMT, bool SPLIT, typename F> cudaError_t pick_kernel(const GemmArgs& a, mx_dtype xdt, int nt, F f) {
    if (a.X)
        return with_dtype(xdt, [&](auto* tp) {
            return with_kernel<FMT, 16, SPLIT, std::remove_pointer_t<decltype(tp)>>(f);
        });
    if (nt == 64) return with_kernel<FMT, 64, SPLIT, void>(f);
    if (nt == 128) return with_kernel<FMT, 128, SPLIT, void>(f);
    return with_kernel<FMT, 16, SPLIT, void>(f);
}

}  // namespace

cudaError_t stream_prepare() {
    auto f = [](auto* kernel, size_t smem, int) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    };
    cudaError_t e = every_kernel<MX_FP4_E4M3_16, false>(f);
    if (e == cudaSuccess) e = every_kernel<MX_FP4_E4M3_16, true>(f);
    if (e == cudaSuccess) e = every_kernel<MX_FP4_E8M0_32, false>(f);
    if (e == cudaSuccess) e = every_kernel<MX_FP4_E8M0_32, true>(f);
    return e;
}

cudaError_t stream_clusters(int split, int* n) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(split);
    cfg.blockDim = dim3(kFusedThreads);
    cfg.dynamicSmemBytes = stream_smem<MX_FP4_E4M3_16, 16, true, true>();
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(n, fp4_stream_kernel<MX_FP4_E4M3_16, 16, true, float>, &cfg);
}

cudaError_t launch_stream(int format, const GemmArgs& a, mx_dtype xdt, int nt, int split, int clusters,
                          bool dependent, cudaStream_t s) {
    auto f = [&](auto* kernel, size_t smem, int threads) {
        return launch_ex(kernel, dim3(clusters * split), dim3(threads), smem, split, dependent, s, a);
    };
    if (format == MX_FP4_E4M3_16)
        return split > 1 ? pick_kernel<MX_FP4_E4M3_16, true>(a, xdt, nt, f)
                         : pick_kernel<MX_FP4_E4M3_16, false>(a, xdt, nt, f);
    return split > 1 ? pick_kernel<MX_FP4_E8M0_32, true>(a, xdt, nt, f)
                     : pick_kernel<MX_FP4_E8M0_32, false>(a, xdt, nt, f);
}

}  // namespace fp4
}  // namespace mx
