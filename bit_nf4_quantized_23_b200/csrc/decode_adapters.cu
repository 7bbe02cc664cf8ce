// Forward of up to 128 tokens, each with its own adapter, over one quantized weight: the decode step
// of many requests (one token each, drafted tokens, or short prompts).
//
//     Y[m] = X[m] W_hat^T + s_a (X[m] A_a^T) B_a^T,   a = adapter_idx[m]
//
// The products with the long reduction over K run in one persistent kernel: D[token, row] with the
// tokens as the MMA's M (128 TMEM lanes, those past M never read) and 256 rows as its N, which takes
// half the MMA instructions that rows as M would.  The rows are first those of A_all of the adapters that
// the batch uses (found by every CTA from the M indices), then those of W_hat.  An adapter's rows meet
// every token and only the products with its own are read, which costs tensor-core time that is idle
// here, and no token meets another's adapter in a sum.
//
// Work units are 256 rows x 64 of K; the units, tile major, are cut into equal contiguous ranges, one
// per CTA (one CTA per SM), and every (tile, CTA) piece is a segment accumulated in TMEM and written as
// an fp32 partial tile to slot tile + CTA.  rows_fixup sums each tile's slots in CTA order, adds the
// adapter term s_a U B_a^T in fp32 and writes Y.
//
// The expansion of the codes bounds the kernel (byte permutes, about three ALU operations a weight on a
// pipe of 64 a clock), so the other roles are kept short: a producer thread expands two blocks of 64
// weights per handshake, the codes' stages are freed as soon as they are in registers, and a unit takes
// four MMAs and two copies.
// Roles (576 threads): warp 0 TMA, warp 1 TMEM owner + MMA issuer, warps 2-17 four groups of producer
// warps that take units in turn; groups 0 and 1 also run the epilogues of even and odd segments.
//
// A parity wait tells apart only neighbouring phases, so no role may come to a barrier two phases
// behind: each group has a row stage and a code stage of its own, an accumulator belongs to one group's
// epilogues, the TMA warp waits for row stages only in the units that begin the range, and the MMA warp
// sees every unit.
#include <algorithm>
#include <climits>

#include "gemm_tc.cuh"
#include "nf4_expand.cuh"
#include "qlora_internal.cuh"
#include "tc_ptx.cuh"

namespace qlora {
namespace {

constexpr int kGroups = 4;
constexpr int kThreads = 64 + 128 * kGroups;
constexpr int kMaxCtas = 256;
constexpr uint32_t kRowStage = 256 * 128;         // 256 rows x 64 16-bit elements
constexpr uint32_t kCodeStage = 256 * 32;         // their packed codes, 32-byte swizzled
constexpr uint32_t kMaxSmem = 227 * 1024;
constexpr int kPrefetch = 2;                      // block constants are loaded this many units (of the group) ahead

struct RowsLayout {
    uint32_t x_stage, off_x, off_codes, off_ids, off_list, off_bars, off_slot, off_abort, off_ballots, alloc;
};
__host__ __device__ inline RowsLayout rows_layout(uint32_t nt, uint32_t xs) {
    RowsLayout l;
    l.x_stage = nt * 128u;                        // X of a unit, [nt x 64], 128-byte swizzled rows
    l.off_x = kGroups * kRowStage;
    // the MMA reads 128 token rows from a stage's start: past the last stage it reads codes
    l.off_codes = l.off_x + xs * l.x_stage;
    l.off_ids = l.off_codes + kGroups * kCodeStage;   // adapter of each token [128]
    l.off_list = l.off_ids + 128 * 4;             // adapters that the batch uses [128]
    l.off_bars = l.off_list + 128 * 4;
    l.off_slot = l.off_bars + (2 * xs + 4 * kGroups + 5) * 8;
    l.off_abort = l.off_slot + 4;
    l.off_ballots = l.off_abort + 4;
    l.alloc = l.off_ballots + 16 + 1024;
    return l;
}

struct RowsParams {
    int32_t M, r, rp;                             // rp: rows an adapter takes, r rounded up to 8
    int32_t steps;                                // units per tile: K / 64
    int32_t w_tiles;                              // tiles of W_hat rows
    int64_t N, K;
    const int32_t* idx;
    int32_t n_adapters;
    const uint8_t* c1_codes;
    const float* c2;
    const float* mu;
    const float* c1f;
    int32_t f16;
    uint32_t nt, x_stages;
    float* partial;                               // [tiles + CTAs][nt][256]
    int32_t* meta;                                // [0] adapters in use, [1 + m] place of token m's adapter among them, or -1
    uint32_t* err;
    NF4Tables tb;
};

__host__ __device__ __forceinline__ int64_t range_begin(int64_t b, int64_t units, int64_t G) { return b * units / G; }

// Adapters whose rows share a tile of A_all rows.
__host__ __device__ __forceinline__ int adapters_per_tile(int rp) { return 256 / rp; }

__global__ void __launch_bounds__(kThreads, 1)
tc_rows_nf4(const __grid_constant__ CUtensorMap tmCodes, const __grid_constant__ CUtensorMap tmX,
            const __grid_constant__ CUtensorMap tmA, RowsParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - ptx::smem_addr(smem_raw));
    const int XS = (int)p.x_stages;
    const RowsLayout lay = rows_layout(p.nt, p.x_stages);
    const uint32_t sB = base, sX = base + lay.off_x, sCodes = base + lay.off_codes;
    int32_t* ids = reinterpret_cast<int32_t*>(gbase + lay.off_ids);
    int32_t* list = reinterpret_cast<int32_t*>(gbase + lay.off_list);
    const uint32_t bar_xfull = base + lay.off_bars, bar_xempty = bar_xfull + 8 * XS;
    const uint32_t bar_cfull = bar_xempty + 8 * XS, bar_cempty = bar_cfull + 8 * kGroups;
    const uint32_t bar_bfull = bar_cempty + 8 * kGroups, bar_bempty = bar_bfull + 8 * kGroups;
    const uint32_t bar_accfull = bar_bempty + 8 * kGroups, bar_accempty = bar_accfull + 16, bar_drain = bar_accempty + 16;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + lay.off_slot);
    volatile int* abort = reinterpret_cast<volatile int*>(gbase + lay.off_abort);
    volatile uint32_t* ballots = reinterpret_cast<volatile uint32_t*>(gbase + lay.off_ballots);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;

    allow_dependents();
    if (tid == 0) {
        for (int s = 0; s < XS; ++s) {
            ptx::mbar_init(bar_xfull + 8 * s, 1);
            ptx::mbar_init(bar_xempty + 8 * s, 1);
        }
        for (int g = 0; g < kGroups; ++g) {
            ptx::mbar_init(bar_cfull + 8 * g, 1);
            ptx::mbar_init(bar_cempty + 8 * g, 4);
            ptx::mbar_init(bar_bfull + 8 * g, 4);
            ptx::mbar_init(bar_bempty + 8 * g, 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(bar_accfull + 8 * a, 1);
            ptx::mbar_init(bar_accempty + 8 * a, 4);
        }
        ptx::mbar_init(bar_drain, 1);
        *abort = 0;
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_smem();
        ptx::tma_prefetch_map(&tmCodes);
        ptx::tma_prefetch_map(&tmX);
        ptx::tma_prefetch_map(&tmA);
    }
    if (warp == 1) {
        ptx::tmem_alloc(base + lay.off_slot, 512);
        ptx::tmem_relinquish();
    }
    grid_dependency_wait();                                   // inputs written by the previous kernel

    // the adapters that the batch uses, in order of first appearance
    int32_t a = -1;
    if (tid < 128) {
        a = tid < p.M ? p.idx[tid] : -1;
        if (a >= p.n_adapters) {
            if (blockIdx.x == 0) atomicOr(p.err, ERR_FLAG_BOUNDS);
            a = -1;
        }
        ids[tid] = a < 0 ? -1 : a;
    }
    __syncthreads();
    int first = tid;
    if (tid < 128) {
        for (int j = (min(tid, p.M) - 1) & ~3; j >= 0; j -= 4) {   // ids past the batch are -1
            const int4 v = *reinterpret_cast<const int4*>(ids + j);
            const int f = v.x == a ? j : v.y == a ? j + 1 : v.z == a ? j + 2 : v.w == a ? j + 3 : 128;
            first = min(first, f);
        }
        const uint32_t b = __ballot_sync(0xffffffffu, a >= 0 && first == tid);
        if (lane == 0) ballots[warp] = b;
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int used = __popc(ballots[0]) + __popc(ballots[1]) + __popc(ballots[2]) + __popc(ballots[3]);
    auto place_of = [&](int t) {                              // of the adapter that first appears at token t
        int n = __popc(ballots[t >> 5] & ((1u << (t & 31)) - 1u));
        for (int w = 0; w < (t >> 5); ++w) n += __popc(ballots[w]);
        return n;
    };
    if (tid < 128) {
        const int place = a >= 0 ? place_of(first) : -1;
        if (a >= 0 && first == tid) list[place] = a;
        if (blockIdx.x == 0) {
            if (tid < p.M) p.meta[1 + tid] = place;
            if (tid == 0) p.meta[0] = used;
        }
    }
    __syncthreads();

    const int S = p.steps;
    const int per_tile = adapters_per_tile(p.rp);
    const int u_tiles = (used + per_tile - 1) / per_tile;     // tiles of A_all rows come first
    const int64_t units = (int64_t)(u_tiles + p.w_tiles) * S;
    const int64_t u0 = range_begin(blockIdx.x, units, gridDim.x);
    const int n = (int)(range_begin(blockIdx.x + 1, units, gridDim.x) - u0);
    const int t0 = (int)(u0 / S), step0 = (int)(u0 - (int64_t)t0 * S);
    const int nu = (int)max((int64_t)0, min((int64_t)n, (int64_t)u_tiles * S - u0));   // units of A_all rows

    if (warp == 0) {
        // unit i: X into token slot i % XS once the MMA that read it before has completed, with it an
        // A_all unit's rows into row stage i % 4; the codes of a W_hat unit into code stage i % 4 once its
        // group has read the last ones
        bool ok = true;
        int issued = 0, tile = t0, step = step0, xs = 0, g = 0;
        uint32_t xph = 1, gph = 1;
        for (int i = 0; i < n && ok; ++i) {
            const bool is_w = i >= nu;
            if (is_w) {
                // stages that A_all units passed over have seen no phase: their first wait passes
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_cempty + 8 * g, (uint32_t)((i - nu) / kGroups + 1) & 1u,
                                                             abort, p.err));
                if (!ok) break;
                if (ptx::elect_one_sync()) {
                    ptx::mbar_arrive_expect_tx(bar_cfull + 8 * g, kCodeStage);
                    ptx::tma_load_2d(sCodes + g * kCodeStage, &tmCodes, step * 32, (tile - u_tiles) * 256, bar_cfull + 8 * g);
                }
                __syncwarp();
            }
            bool w = ptx::mbar_wait(bar_xempty + 8 * xs, xph, abort, p.err);
            if (w && !is_w) w = ptx::mbar_wait(bar_bempty + 8 * g, gph, abort, p.err);
            ok = __all_sync(0xffffffffu, w);
            if (ok && ptx::elect_one_sync()) {
                const uint32_t fb = bar_xfull + 8 * xs;
                const int ad0 = tile * per_tile, ads = is_w ? 0 : min(per_tile, used - ad0);
                ptx::mbar_arrive_expect_tx(fb, lay.x_stage + (uint32_t)(ads * p.rp) * 128u);
                ptx::tma_load_2d(sX + xs * lay.x_stage, &tmX, step * 64, 0, fb);
                for (int q = 0; q < ads; ++q)
                    ptx::tma_load_3d(sB + g * kRowStage + (uint32_t)(q * p.rp) * 128u, &tmA, step * 64, 0, list[ad0 + q], fb);
            }
            __syncwarp();
            issued = ok ? i + 1 : i;
            if (++step == S) { step = 0; ++tile; }
            if (++xs == XS) { xs = 0; xph ^= 1u; }
            if (++g == kGroups) { g = 0; gph ^= 1u; }
        }
        if (*abort) {   // drain this CTA's copies in flight before it exits
            for (int c = max(0, issued - XS); c < issued; ++c)
                ptx::mbar_wait_drain(bar_xfull + 8 * (c % XS), (uint32_t)(c / XS) & 1u);
            // the codes of the unit after the last token tile may be in flight too
            const int end = min(issued + 1, n);
            for (int c = max(nu, end - kGroups); c < end; ++c)
                ptx::mbar_wait_drain(bar_cfull + 8 * (c % kGroups), (uint32_t)((c - nu) / kGroups) & 1u);
        }
    } else if (warp == 1) {
        const uint32_t idesc = ptx::idesc_set_f16(ptx::idesc_bf16_f32_ab(128, 256, 0, 0), p.f16 != 0);
        const uint64_t x_sw = ptx::smem_desc_sw128(sX, 16, 1024);
        const uint64_t b_none = ptx::smem_desc_kmajor_none(sB, 256 * 16, 128);   // W_hat rows, as the producers write them
        const uint64_t b_sw = ptx::smem_desc_sw128(sB, 16, 1024);                // A_all rows, as TMA does
        bool ok = true, fresh = true;
        int step = step0, xs = 0, g = 0;
        uint32_t xph = 0, gph = 0, acc = 0, acc_ph = 1;       // accumulator of the segment at hand and its use, mod 2
        for (int i = 0; i < n && ok; ++i) {
            if (fresh) {                                      // drained by the epilogue of its last segment
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_accempty + 8 * acc, acc_ph, abort, p.err));
                if (!ok) break;
            }
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_xfull + 8 * xs, xph, abort, p.err) &&
                                             ptx::mbar_wait(bar_bfull + 8 * g, gph, abort, p.err));
            if (!ok) break;
            ptx::tc_fence_after();
            const bool last = (step + 1 == S) || (i == n - 1);
            if (ptx::elect_one_sync()) {
                const bool is_w = i >= nu;
                const uint64_t ad = x_sw + (uint32_t)xs * (lay.x_stage >> 4);
                const uint64_t bd = (is_w ? b_none : b_sw) + (uint32_t)g * (kRowStage >> 4);
                const uint32_t bk = is_w ? (2u * 256 * 16) >> 4 : 32u >> 4, d = tmem + 256u * acc;
                ptx::mma_bf16_ss(d, ad, bd, idesc, fresh ? 0u : 1u);
                ptx::mma_bf16_ss(d, ad + 2, bd + bk, idesc, 1u);
                ptx::mma_bf16_ss(d, ad + 4, bd + 2 * bk, idesc, 1u);
                ptx::mma_bf16_ss(d, ad + 6, bd + 3 * bk, idesc, 1u);
                ptx::mma_commit(bar_bempty + 8 * g);
                ptx::mma_commit(bar_xempty + 8 * xs);
                if (last) ptx::mma_commit(bar_accfull + 8 * acc);   // the segment ends: hand the accumulator over
            }
            __syncwarp();
            if (++xs == XS) { xs = 0; xph ^= 1u; }
            if (++g == kGroups) { g = 0; gph ^= 1u; }
            fresh = last;
            if (++step == S) step = 0;
            if (last) {
                acc ^= 1u;
                if (acc == 0) acc_ph ^= 1u;
            }
        }
        if (ptx::elect_one_sync()) {
            ptx::mma_commit(bar_drain);
            if (*abort) ptx::mbar_wait_drain(bar_drain, 0);   // issued MMAs finish before TMEM is freed
        }
        __syncwarp();
    } else {
        // group g takes units g, g + 4, ...; thread t expands rows t and t + 128 of the unit's tile
        const int g = (warp - 2) >> 2, t = tid - 64 - 128 * g;
        const float mu = p.c1f ? 0.f : *p.mu;
        // block constants of a unit, as loaded (any arithmetic here would wait for the loads): the E4M3
        // codes (or fp32 constants) of its two blocks and their c2.  `at` is the block index of row t.
        struct Cursor { int tile, step; int64_t at; };
        const int64_t kb = S;                                 // blocks per W row
        auto place = [&](Cursor& c) { c.at = ((int64_t)(c.tile - u_tiles) * 256 + t) * kb + c.step; };
        auto advance = [&](Cursor& c) {
            c.step += kGroups;
            c.at += kGroups;
            if (c.step >= S) {
                while (c.step >= S) { c.step -= S; ++c.tile; }
                place(c);
            }
        };
        const int64_t half = 128 * kb, nb1 = p.N * kb;        // a row exists when its blocks do
        struct Consts { uint32_t ca, cb; float c2a, c2b; };
        auto load_consts = [&](const Cursor& c) {
            Consts k{0, 0, 0.f, 0.f};
            if (c.tile < u_tiles) return k;
            const bool two = c.at + half < nb1;
            if (c.at >= nb1) return k;
            if (p.c1f) {
                k.c2a = __ldg(p.c1f + c.at);
                if (two) k.c2b = __ldg(p.c1f + c.at + half);
            } else {
                k.ca = __ldg(p.c1_codes + c.at);
                k.c2a = __ldg(p.c2 + (c.at >> 8));
                if (two) {
                    k.cb = __ldg(p.c1_codes + c.at + half);
                    k.c2b = __ldg(p.c2 + ((c.at + half) >> 8));
                }
            }
            return k;
        };
        Cursor cur{t0, step0 + g, 0};
        while (cur.step >= S) { cur.step -= S; ++cur.tile; }
        place(cur);
        Cursor pf = cur;
        Consts q[kPrefetch];
#pragma unroll
        for (int d = 0; d < kPrefetch; ++d) {
            q[d] = Consts{0, 0, 0.f, 0.f};
            if (g + kGroups * d < n) q[d] = load_consts(pf);
            advance(pf);
        }

        int epi_seg = g < 2 ? g : INT_MAX / 2;                // next segment whose epilogue is this group's
        const int last_seg = (int)((u0 + n - 1) / S) - t0;
        auto epilogue = [&](int seg) -> bool {
            const bool ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_accfull + 8 * g, (uint32_t)(seg >> 1) & 1u,
                                                                    abort, p.err));
            if (!ok) return false;
            ptx::tc_fence_after();
            const uint32_t quad = (uint32_t)(warp & 3);       // TMEM lanes that the warp reaches: its tokens
            const int m = (int)(quad * 32u) + lane;
            if ((int)(quad * 32u) < p.M) {
                float* dst = p.partial + ((int64_t)(t0 + seg + blockIdx.x) * p.nt + m) * 256;
#pragma unroll 1
                for (uint32_t c = 0; c < 256; c += 32) {
                    uint32_t v[32];
                    ptx::tmem_ld_32x32b_x32(tmem + ((quad * 32u) << 16) + 256u * (uint32_t)g + c, v);
                    ptx::tmem_ld_wait();
                    if (m < p.M) {
                        uint4* d4 = reinterpret_cast<uint4*>(dst + c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) d4[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_accempty + 8 * g);
            return true;
        };

        bool ok = true;
        uint32_t cph = 0, ph = 1;
        for (int i = g; i < n && ok; i += kGroups) {
            const int seg = cur.tile - t0;
            while (epi_seg < seg && ok) { ok = epilogue(epi_seg); epi_seg += 2; }
            if (!ok) break;
            const Consts k = q[0];
#pragma unroll
            for (int d = 0; d + 1 < kPrefetch; ++d) q[d] = q[d + 1];
            q[kPrefetch - 1] = Consts{0, 0, 0.f, 0.f};
            if (i + kGroups * kPrefetch < n) q[kPrefetch - 1] = load_consts(pf);
            if (i >= nu) {
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_cfull + 8 * g, cph, abort, p.err));
                if (!ok) break;
                cph ^= 1u;
                const uint32_t src = sCodes + g * kCodeStage + (uint32_t)t * 32u, swz = (((uint32_t)t >> 2) & 1u) << 4;
                uint4 w[4];
                w[0] = ld_shared_v4(src + swz);
                w[1] = ld_shared_v4(src + (16u ^ swz));
                w[2] = ld_shared_v4(src + 4096u + swz);
                w[3] = ld_shared_v4(src + 4096u + (16u ^ swz));
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar_cempty + 8 * g);   // the codes are in registers
                Lut lut;
                // rows past N have a constant of 0 and so expand to zeros
                float c1p = p.c1f ? k.c2a : __fadd_rn(__fmul_rn(e4m3_to_f32(k.ca), k.c2a), mu);
                if (cur.at >= nb1) c1p = 0.f;
                build_lut(lut, c1p, p.tb, p.f16 != 0);
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_bempty + 8 * g, ph, abort, p.err));
                if (!ok) break;
                const uint32_t dst = sB + g * kRowStage + (uint32_t)t * 16u;
                expand_block_row_kn<256 * 16>(dst, w[0], w[1], lut);
                c1p = p.c1f ? k.c2b : __fadd_rn(__fmul_rn(e4m3_to_f32(k.cb), k.c2b), mu);
                if (cur.at + half >= nb1) c1p = 0.f;
                build_lut(lut, c1p, p.tb, p.f16 != 0);
                expand_block_row_kn<256 * 16>(dst + 128u * 16u, w[2], w[3], lut);
                ptx::fence_proxy_async_smem();
            } else {                                          // TMA brings the rows; keep the stage's phases
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_bempty + 8 * g, ph, abort, p.err));
                if (!ok) break;
            }
            ph ^= 1u;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_bfull + 8 * g);
            advance(cur);
            advance(pf);
        }
        while (ok && epi_seg <= last_seg) { ok = epilogue(epi_seg); epi_seg += 2; }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// Y[m, n] = the sum of the partial tiles of n / 256 in CTA order + sum_j (s_a U[m, j]) B_a[n, j] (fp32),
// rounded to the output type.  CTA (tile, y): the tile's 256 columns and the y-th 8 or 16 tokens; a thread has
// one column and half of the tokens.  The kernel is a chain of memory latencies, so each link has all its
// loads in flight: the B rows of the CTA's tokens come by cp.async, 32 KiB at a time, while U is summed
// from its own partial tiles and the base product from its slots.  Neighbouring tokens of one request
// are a run and share B.
constexpr int kFixThreads = 512;
constexpr int kFixLoads = 16;                     // loads of partial sums that a thread has in flight together
constexpr int kFixChunks = 8;                     // 16-byte chunks (8 ranks) of B per column and pass, over all runs

struct FixParams {
    const float* partial;
    const int32_t* meta;
    const int32_t* idx;
    const float* scales;
    const uint16_t* B;
    float* U;
    void* out;
    int64_t N;
    int32_t M, r, rp, steps, w_tiles, G;
    uint32_t nt;
    int32_t out_f32, f16;
};

__host__ __device__ inline uint32_t fixup_smem(int r, int tokens) {
    return kFixChunks * 256 * 16 + (uint32_t)tokens * (uint32_t)((r + 7) / 8 * 8) * 4;
}

// kFixOwn: tokens of a thread; a CTA has twice as many.
template <int kFixOwn>
__global__ void __launch_bounds__(kFixThreads, 2)
rows_fixup(FixParams p) {
    constexpr int kFixTokens = 2 * kFixOwn, kFixSlots = kFixLoads / kFixOwn;
    extern __shared__ __align__(16) uint8_t smem[];
    uint4* bs = reinterpret_cast<uint4*>(smem);               // bs[(run * pass_chunks + c) * 256 + column]
    float* us = reinterpret_cast<float*>(smem + kFixChunks * 256 * 16);   // us[q * pitch + j] = s_a U[m0 + q, j]
    __shared__ int32_t tok_place[kFixTokens], tok_adapter[kFixTokens], tok_run[kFixTokens], run_adapter[kFixTokens];
    __shared__ int32_t runs_of;
    __shared__ int2 span[129];                                // first and last CTA of each tile of A_all rows; [128]: this tile's
    const int tid = threadIdx.x, col = tid & 255, q0 = (tid >> 8) * kFixOwn;
    const int m0 = (int)blockIdx.y * kFixTokens, nm = min(p.M - m0, kFixTokens);
    grid_dependency_wait();                                   // partial tiles are complete
    const int per_tile = adapters_per_tile(p.rp);
    const int u_tiles = (p.meta[0] + per_tile - 1) / per_tile;
    const int64_t units = (int64_t)(u_tiles + p.w_tiles) * p.steps;
    const int64_t slot_floats = (int64_t)p.nt * 256;
    const int tile = u_tiles + (int)blockIdx.x;
    // the CTA whose range holds unit u: the largest b with b units / G <= u, that is b units < (u + 1) G
    auto cta_of = [&](int64_t u) { return (int)(((u + 1) * p.G - 1) / units); };
    auto span_of = [&](int t) {
        return make_int2(cta_of((int64_t)t * p.steps), cta_of((int64_t)t * p.steps + p.steps - 1));
    };
    if (tid >= 256 && tid - 256 < u_tiles) span[tid - 256] = span_of(tid - 256);
    if (tid == 128) span[128] = span_of(tile);
    if (tid < 32) {                                           // tokens, and the runs of equal adapters among them
        const int place = tid < nm ? p.meta[1 + m0 + tid] : -1;
        const int a = place >= 0 ? p.idx[m0 + tid] : -1;
        const int before = __shfl_up_sync(0xffffffffu, a, 1);
        const uint32_t starts = __ballot_sync(0xffffffffu, a >= 0 && (tid == 0 || a != before));
        const int run = __popc(starts & (0xffffffffu >> (31 - tid))) - 1;
        if (tid < kFixTokens) {
            tok_place[tid] = place;
            tok_adapter[tid] = a;
            tok_run[tid] = a >= 0 ? run : -1;
            if (starts >> tid & 1u) run_adapter[run] = a;
        }
        if (tid == 0) runs_of = __popc(starts);
    }
    __syncthreads();
    const int runs = runs_of, all_chunks = (p.r + 7) / 8, pitch = all_chunks * 8;
    // runs and chunks of B that are in shared memory together
    const int pass_runs = min(runs, kFixChunks), pass_chunks = runs > 0 ? min(all_chunks, kFixChunks / pass_runs) : 0;
    const int64_t n = (int64_t)blockIdx.x * 256 + col;
    const bool in = n < p.N;
    auto fetch = [&](int r0, int c0) {                        // B chunks c0 .. of runs r0 ..
        const int nr = min(pass_runs, runs - r0), nc = min(pass_chunks, all_chunks - c0);
        for (int e = tid >> 8; e < nr * nc && in; e += 2) {
            const int run = e / nc, c = e - run * nc;
            const uint16_t* src = p.B + ((int64_t)run_adapter[r0 + run] * p.N + n) * p.r + (c0 + c) * 8;
            uint4* dst = bs + (run * pass_chunks + c) * 256 + col;
            if ((p.r & 7) == 0) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_addr(dst)), "l"(src) : "memory");
            } else {                                          // rows of B start anywhere
                uint32_t v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = (c0 + c) * 8 + i < p.r ? src[i] : 0u;
                *dst = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
            }
        }
    };
    fetch(0, 0);

    // the base product: .x starts with it and takes the even ranks' terms, .y the odd ones'
    float2 acc[kFixOwn];
#pragma unroll
    for (int q = 0; q < kFixOwn; ++q) acc[q] = make_float2(0.f, 0.f);
    {
        const int2 sp = span[128];
        const float* src = p.partial + (int64_t)(tile + sp.x) * slot_floats + (int64_t)(m0 + q0) * 256 + col;
        for (int b = sp.x; b <= sp.y; b += kFixSlots, src += kFixSlots * slot_floats) {
            float v[kFixSlots][kFixOwn];
#pragma unroll
            for (int e = 0; e < kFixSlots; ++e)
#pragma unroll
                for (int q = 0; q < kFixOwn; ++q)
                    v[e][q] = q0 + q < nm && b + e <= sp.y ? src[e * slot_floats + q * 256] : 0.f;
#pragma unroll
            for (int e = 0; e < kFixSlots; ++e)
#pragma unroll
                for (int q = 0; q < kFixOwn; ++q) acc[q].x = __fadd_rn(acc[q].x, v[e][q]);
        }
    }
    for (int i = tid; i < kFixTokens * pitch; i += kFixThreads) {
        const int q = i / pitch, j = i - q * pitch;
        float v = 0.f, sc = 0.f;
        if (j < p.r && tok_place[q] >= 0) {
            sc = __ldg(p.scales + tok_adapter[q]);
            const int t = tok_place[q] / per_tile, row = (tok_place[q] - t * per_tile) * p.rp + j;
            const int2 sp = span[t];
            const float* src = p.partial + (int64_t)(t + sp.x) * slot_floats + (int64_t)(m0 + q) * 256 + row;
            for (int b = sp.x; b <= sp.y; b += 8, src += 8 * slot_floats) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = b + e <= sp.y ? src[e * slot_floats] : 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) v = __fadd_rn(v, x[e]);
            }
        }
        us[i] = __fmul_rn(sc, v);
        if (p.U && blockIdx.x == 0 && q < nm && j < p.r) p.U[(int64_t)(m0 + q) * p.r + j] = v;
    }

    const bool f16 = p.f16 != 0;
    for (int r0 = 0; r0 < runs; r0 += pass_runs) {
        for (int c0 = 0; c0 < all_chunks; c0 += pass_chunks) {
            if (r0 > 0 || c0 > 0) {
                __syncthreads();                              // the last pass has been read
                fetch(r0, c0);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();                                  // us and every thread's copies
            const int nc = min(pass_chunks, all_chunks - c0);
            for (int c = 0; c < nc; ++c) {
                int have = -1;
                float2 bv[4];
#pragma unroll
                for (int q = 0; q < kFixOwn; ++q) {
                    const int run = tok_run[q0 + q] - r0;
                    if (run < 0 || run >= pass_runs) continue;
                    if (run != have) {
                        have = run;
                        const uint4 w = bs[(run * pass_chunks + c) * 256 + col];
                        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            bv[e] = make_float2(from16(x[e] & 0xFFFFu, f16), from16(x[e] >> 16, f16));
                    }
                    const float4* u4 = reinterpret_cast<const float4*>(us + (q0 + q) * pitch + (c0 + c) * 8);
                    const float4 u0 = u4[0], u1 = u4[1];
                    acc[q] = fma2_rn(make_float2(u0.x, u0.y), bv[0], acc[q]);
                    acc[q] = fma2_rn(make_float2(u0.z, u0.w), bv[1], acc[q]);
                    acc[q] = fma2_rn(make_float2(u1.x, u1.y), bv[2], acc[q]);
                    acc[q] = fma2_rn(make_float2(u1.z, u1.w), bv[3], acc[q]);
                }
            }
        }
    }
    if (!in) return;
#pragma unroll
    for (int q = 0; q < kFixOwn; ++q) {
        if (q0 + q >= nm) break;
        const int64_t at = (int64_t)(m0 + q0 + q) * p.N + n;
        const float y = __fadd_rn(acc[q].x, acc[q].y);
        if (p.out_f32) static_cast<float*>(p.out)[at] = y;
        else static_cast<uint16_t*>(p.out)[at] = (uint16_t)to16_rn(y, f16);
    }
}

// ---------------------------------------------------------------------------- host

inline int32_t adapter_rows(int32_t r) { return (r + 7) / 8 * 8; }

template <int OWN>
qlora_status launch_fixup(const FixParams& f, cudaStream_t stream) {
    static bool configured = false;   // attribute set once per instantiation (idempotent, so races are benign)
    if (!configured) {
        if (cudaFuncSetAttribute(rows_fixup<OWN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)fixup_smem(256, 2 * OWN)) != cudaSuccess)
            return QLORA_ERR_CUDA;
        configured = true;
    }
    const dim3 grid((unsigned)f.w_tiles, (unsigned)((f.M + 2 * OWN - 1) / (2 * OWN)));
    (void)launch_dependent(rows_fixup<OWN>, grid, dim3(kFixThreads), fixup_smem(f.r, 2 * OWN), stream, f);
    QLORA_CHECK_LAUNCH();
    return QLORA_OK;
}

inline uint32_t token_tile(int64_t M) { return (uint32_t)((M + 7) / 8 * 8); }

}  // namespace

// meta [1 + 128] int32, then the partial tiles of every W tile and of the tiles of A_all rows that M
// tokens can use, plus one for each CTA boundary.
size_t rows_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t r, int64_t n_adapters) {
    const int64_t per_tile = adapters_per_tile(adapter_rows(r));
    const int64_t tiles = (N + 255) / 256 + (std::min(M, n_adapters) + per_tile - 1) / per_tile;
    return 1024 + (size_t)(tiles + kMaxCtas) * token_tile(M) * 256 * sizeof(float);
}

qlora_status launch_rows(const RowsArgs& a, cudaStream_t stream) {
    const qlora_nf4_weight* w = a.w;
    const int64_t N = w->N, K = w->K;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return QLORA_ERR_CUDA;
    static bool configured = false;
    if (!configured) {
        if (cudaFuncSetAttribute(tc_rows_nf4, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem) != cudaSuccess)
            return QLORA_ERR_CUDA;
        configured = true;
    }
    RowsParams p{};
    p.M = (int32_t)a.M; p.r = a.r;
    p.rp = adapter_rows(a.r);
    p.steps = (int32_t)(K / 64);
    p.w_tiles = (int32_t)((N + 255) / 256);
    p.N = N; p.K = K;
    p.idx = a.idx; p.n_adapters = a.n_adapters;
    p.c1_codes = w->c1_codes; p.c2 = w->c2; p.mu = w->mu; p.c1f = w->c1;
    p.f16 = w->compute_dtype == QLORA_DTYPE_F16;
    p.nt = token_tile(a.M);
    p.x_stages = 6;                                           // as many token stages as fit, up to six
    while (p.x_stages > 2 && rows_layout(p.nt, p.x_stages).alloc > kMaxSmem) --p.x_stages;
    const RowsLayout lay = rows_layout(p.nt, p.x_stages);
    if (lay.alloc > kMaxSmem) return QLORA_ERR_UNSUPPORTED;
    p.meta = static_cast<int32_t*>(a.workspace);
    p.partial = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + 1024);
    p.tb = host_tables(w->codebook);
    p.err = device_error_word();
    if (!p.err) return QLORA_ERR_CUDA;
    CUtensorMap tmCodes, tmX, tmA;
    if (!make_tmap_codes32(&tmCodes, w->codes, K / 2, N)) return QLORA_ERR_CUDA;
    if (!make_tmap_3d(&tmA, a.A, K, a.r, a.n_adapters, 64, (uint32_t)p.rp)) return QLORA_ERR_CUDA;
    if (!make_tmap_2d(&tmX, true, a.X, K, a.M, K * 2, 64, p.nt, true)) return QLORA_ERR_CUDA;
    const int64_t G = std::min<int64_t>({(int64_t)p.w_tiles * p.steps, (int64_t)sms, (int64_t)kMaxCtas});
    (void)launch_dependent(tc_rows_nf4, dim3((unsigned)G), dim3(kThreads), lay.alloc, stream, tmCodes, tmX, tmA, p);
    QLORA_CHECK_LAUNCH();
    FixParams f{};
    f.partial = p.partial; f.meta = p.meta; f.idx = a.idx; f.scales = a.scales;
    f.B = static_cast<const uint16_t*>(a.B); f.U = a.U; f.out = a.out; f.N = N;
    f.M = p.M; f.r = p.r; f.rp = p.rp; f.steps = p.steps; f.w_tiles = p.w_tiles; f.G = (int32_t)G; f.nt = p.nt;
    f.out_f32 = a.out_f32; f.f16 = p.f16;
    // tokens of a fix-up CTA: 8 for the shortest chain of latencies, 16 when the tokens would otherwise
    // take several waves of CTAs
    QLORA_TRY(a.M <= 64 ? launch_fixup<4>(f, stream) : launch_fixup<8>(f, stream));
    return QLORA_OK;
}

}  // namespace qlora
