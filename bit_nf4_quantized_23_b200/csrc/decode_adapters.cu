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
// an fp32 partial tile to slot tile + CTA.  The tensor cores' fp32 sums lose about 2^-27 of themselves at
// each step, one way, so tiles of A_all rows, whose U must keep fp32 digits for the gradients, are cut
// into pieces of 1024 of K, each with slots of its own.  Tiles of W_hat rows are not: their sums are as long as a
// CTA's share of the tile, which a Y in fp32 shows.  rows_finish_U sums the adapters' tiles to U, tc_rows_fixup
// the others, adds the adapter term s_a U B_a^T on the tensor cores and writes Y.
//
// The expansion of the codes bounds the kernel (byte permutes, about three ALU operations a weight on a
// pipe of 64 a clock), so the other roles are kept short: a producer thread expands two blocks of 64
// weights per handshake, the codes' stages are freed as soon as they are in registers, and a unit takes
// four MMAs and two copies.
// Roles (608 threads): warp 0 TMA of the tokens (and A_all rows), warp 1 TMEM owner + MMA issuer, warp 2
// TMA of the codes (a warp of its own: behind the token ring the codes came a unit too late, 6% of the forward at
// W[28672, 8192] and 112 tokens), warps 3-18 four groups of producer warps that take units in
// turn; groups 0 and 1 also run the epilogues of even and odd segments.
//
// Times below are of the whole forward, as CUDA graph replays over three weights in turn.
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
constexpr int kThreads = 96 + 128 * kGroups;
constexpr int kMaxCtas = 256;
constexpr uint32_t kRowStage = 256 * 128;         // 256 rows x 64 16-bit elements
constexpr uint32_t kCodeStage = 256 * 32;         // their packed codes, 32-byte swizzled
constexpr uint32_t kMaxSmem = 227 * 1024;
constexpr int kPiece = 16;                        // units of a piece of a tile of A_all rows
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
    int2* piece_ctas;                             // first and last CTA of each piece of A_all rows
    int32_t* meta;                                // [0] adapters in use, [1 + m] place of token m's adapter among them, or -1
    uint32_t* err;
    NF4Tables tb;
};

__host__ __device__ __forceinline__ int64_t range_begin(int64_t b, int64_t units, int64_t G) { return b * units / G; }

// Slots are counted in pieces: a tile of A_all rows has pieces_of(S) of them, a W_hat tile one.
__host__ __device__ __forceinline__ int pieces_of(int S) { return (S + kPiece - 1) / kPiece; }
__device__ __forceinline__ int piece_at(int tile, int step, int u_tiles, int pieces) {
    return tile < u_tiles ? tile * pieces + step / kPiece : u_tiles * pieces + (tile - u_tiles);
}

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
        ids[tid] = place;                                     // from here on the token's place among the adapters
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
    const int pieces = pieces_of(S), piece0 = piece_at(t0, step0, u_tiles, pieces);   // segment s is piece piece0 + s

    if (warp == 0) {
        // unit i: X into token slot i % XS once the MMA that read it before has completed, with it an
        // A_all unit's rows into row stage i % 4
        bool ok = true;
        int issued = 0, tile = t0, step = step0, xs = 0, g = 0;
        uint32_t xph = 1, gph = 1;
        for (int i = 0; i < n && ok; ++i) {
            const bool is_w = i >= nu;
            bool w = ptx::mbar_wait(bar_xempty + 8 * xs, xph, abort, p.err);
            if (w && !is_w) w = ptx::mbar_wait(bar_bempty + 8 * g, gph, abort, p.err);
            ok = __all_sync(0xffffffffu, w);
            if (!ok) break;
            if (ptx::elect_one_sync()) {
                const uint32_t fb = bar_xfull + 8 * xs;
                const int ad0 = tile * per_tile, ads = is_w ? 0 : min(per_tile, used - ad0);
                ptx::mbar_arrive_expect_tx(fb, lay.x_stage + (uint32_t)(ads * p.rp) * 128u);
                ptx::tma_load_2d(sX + xs * lay.x_stage, &tmX, step * 64, 0, fb);
                for (int q = 0; q < ads; ++q)
                    ptx::tma_load_3d(sB + g * kRowStage + (uint32_t)(q * p.rp) * 128u, &tmA, step * 64, 0, list[ad0 + q], fb);
            }
            __syncwarp();
            issued = i + 1;
            if (++step == S) { step = 0; ++tile; }
            if (++xs == XS) { xs = 0; xph ^= 1u; }
            if (++g == kGroups) { g = 0; gph ^= 1u; }
        }
        if (*abort) {   // drain this warp's copies in flight before the CTA exits
            for (int c = max(0, issued - XS); c < issued; ++c)
                ptx::mbar_wait_drain(bar_xfull + 8 * (c % XS), (uint32_t)(c / XS) & 1u);
        }
    } else if (warp == 2) {
        // the codes of W_hat unit i into code stage i % 4 once its group has read the last ones.  Stages that
        // A_all units passed over have seen no phase: their first wait passes.
        bool ok = true;
        int issued = nu;
        int64_t u = u0 + nu;
        int tile = (int)(u / S), step = (int)(u - (int64_t)tile * S), g = nu % kGroups;
        for (int i = nu; i < n && ok; ++i) {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_cempty + 8 * g, (uint32_t)((i - nu) / kGroups + 1) & 1u, abort, p.err));
            if (!ok) break;
            if (ptx::elect_one_sync()) {
                ptx::mbar_arrive_expect_tx(bar_cfull + 8 * g, kCodeStage);
                ptx::tma_load_2d(sCodes + g * kCodeStage, &tmCodes, step * 32, (tile - u_tiles) * 256, bar_cfull + 8 * g);
            }
            __syncwarp();
            issued = i + 1;
            if (++step == S) { step = 0; ++tile; }
            if (++g == kGroups) g = 0;
        }
        if (*abort) {
            for (int c = max(nu, issued - kGroups); c < issued; ++c)
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
            const bool is_w = i >= nu;
            const bool last = (step + 1 == S) || (i == n - 1) || (!is_w && (step + 1) % kPiece == 0);
            if (ptx::elect_one_sync()) {
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
        const int g = (warp - 3) >> 2, t = tid - 96 - 128 * g;
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
        const int t_end = (int)((u0 + n - 1) / S);
        const int last_seg = piece_at(t_end, (int)(u0 + n - 1 - (int64_t)t_end * S), u_tiles, pieces) - piece0;
        auto epilogue = [&](int seg) -> bool {
            const bool ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_accfull + 8 * g, (uint32_t)(seg >> 1) & 1u,
                                                                    abort, p.err));
            if (!ok) return false;
            ptx::tc_fence_after();
            const int piece = piece0 + seg;
            const uint32_t quad = (uint32_t)(warp & 3);       // TMEM lanes that the warp reaches: its tokens
            const int m = (int)(quad * 32u) + lane;
            uint32_t lo = 0, hi = m < p.M ? 256 : 0;          // columns that the token needs
            if (piece < u_tiles * pieces) {                   // of A_all rows only its own adapter's
                const int q = ids[m] - piece / pieces * per_tile;
                lo = (uint32_t)(q * p.rp);
                hi = hi && ids[m] >= 0 && q >= 0 && q < per_tile ? lo + (uint32_t)p.r : 0;
            }
            if (t == 0 && piece < u_tiles * pieces) {         // note the piece's first and last CTA for rows_finish_U
                const int tile = piece / pieces, k = piece - tile * pieces;
                const int64_t begin = (int64_t)tile * S + k * kPiece, end = (int64_t)tile * S + min(S, (k + 1) * kPiece);
                if (begin >= u0) p.piece_ctas[piece].x = (int32_t)blockIdx.x;
                if (end <= u0 + n) p.piece_ctas[piece].y = (int32_t)blockIdx.x;
            }
            if ((int)(quad * 32u) < p.M) {
                float* dst = p.partial + ((int64_t)(piece0 + seg + blockIdx.x) * p.nt + m) * 256;
#pragma unroll 1
                for (uint32_t c = 0; c < 256; c += 32) {
                    uint32_t v[32];
                    ptx::tmem_ld_32x32b_x32(tmem + ((quad * 32u) << 16) + 256u * (uint32_t)g + c, v);
                    ptx::tmem_ld_wait();
                    if (c < hi && c + 32 > lo) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8)       // whole 32-byte sectors: 29.6 to 26 us at 100 tokens, W[1024, 1024]
                            store_sector(dst + c + i, v + i);
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
            const int seg = piece_at(cur.tile, cur.step, u_tiles, pieces) - piece0;
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
                // The codes are in registers before the stage is given up: the loads above are still in flight
                // here, and the copy that follows is the async proxy's, which an arrive alone does not order.
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar_cempty + 8 * g);
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

// The CTAs whose ranges hold the units u .. u + count - 1: unit u belongs to the largest b with
// b units / G <= u, that is b units < (u + 1) G.
__device__ __forceinline__ int2 unit_span(int64_t u, int count, int64_t units, int G) {
    return make_int2((int)(((u + 1) * G - 1) / units), (int)(((u + count) * G - 1) / units));
}

struct FixParams {
    const float* partial;
    const int2* piece_ctas;
    const int32_t* meta;
    const int32_t* idx;
    const float* scales;
    float* U;
    uint16_t* U2;
    void* out;
    int64_t N;
    int32_t M, r, R, rp, steps, w_tiles, G;
    int32_t all_pieces;       // of A_all rows, at most
    uint32_t nt;
    int32_t out_f32, f16, stages;
    uint32_t* err;
};

// U[m, j] = the sum of its partial tiles in CTA order (stored when the caller keeps U), and the hi/lo
// halves of s_a U[m, j] in the 16-bit compute type, U2 [M, 2R]: zeros for j >= r and without an adapter.
__global__ void __launch_bounds__(128)
rows_finish_U(FixParams p) {
    __shared__ int2 ctas[128];                                // of the first pieces: loaded with the tokens' places
    grid_dependency_wait();
    allow_dependents();
    const int i = (int)(blockIdx.x * 128 + threadIdx.x), m = i / p.R, j = i - m * p.R;
    const int place = m < p.M ? p.meta[1 + m] : -1, adapter = m < p.M ? p.idx[m] : -1;
    if ((int)threadIdx.x < p.all_pieces) ctas[threadIdx.x] = p.piece_ctas[threadIdx.x];
    __syncthreads();
    if (m >= p.M) return;
    float v = 0.f, sv = 0.f;
    if (place >= 0 && j < p.r) {
        const float sc = __ldg(p.scales + adapter);
        const int per_tile = adapters_per_tile(p.rp), t = place / per_tile, row = (place - t * per_tile) * p.rp + j;
        const int64_t slot_floats = (int64_t)p.nt * 256;
        const int pieces = pieces_of(p.steps), first = t * pieces;
        const float* src = p.partial + (int64_t)first * slot_floats + (int64_t)m * 256 + row;
        for (int k0 = 0; k0 < pieces; k0 += 4) {              // four pieces' first three slots in flight
            int2 c[4];
            float x[4][3];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = k0 + e;
                c[e] = k >= pieces ? make_int2(0, -1) : first + k < 128 ? ctas[first + k] : p.piece_ctas[first + k];
#pragma unroll
                for (int b = 0; b < 3; ++b) x[e][b] = c[e].x + b <= c[e].y ? src[(k + c[e].x + b) * slot_floats] : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int b = 0; b < 3; ++b) v = __fadd_rn(v, x[e][b]);
                for (int b = c[e].x + 3; b <= c[e].y; ++b) v = __fadd_rn(v, src[(k0 + e + b) * slot_floats]);
            }
        }
        sv = __fmul_rn(sc, v);
    }
    if (p.U && j < p.r) p.U[(int64_t)m * p.r + j] = v;
    const bool f16 = p.f16 != 0;
    const uint32_t hi = to16_rn(sv, f16);
    p.U2[(int64_t)m * 2 * p.R + j] = (uint16_t)hi;
    p.U2[(int64_t)m * 2 * p.R + p.R + j] = (uint16_t)to16_rn(__fsub_rn(sv, from16(hi, f16)), f16);
}

// Y[m, n] = the sum of the partial tiles of n / 256 in CTA order + s_a U[m] B_a[n]^T, rounded to the
// output type.  CTA x: columns 64 x .. 64 x + 63 of every token (128 accumulator rows).  The adapter term
// is the fused GEMM's: hi and lo of s_a U meet the adapter's B on the tensor cores, and the MMAs of one
// adapter write only its tokens' rows.  The four epilogue warps sum the base product meanwhile.
//
// The kernel starts when every CTA of rows_finish_U has seen the rows kernel complete (it lets dependents
// start after its own wait), so only U2 has to be waited for: the partial tiles, the tokens' places and B
// are read at once (48 tokens, W[8192, 8192], the whole forward: 50.7 to 49.5 us).  Such reads pass by L1
// (__ldcg, TMA), which may hold lines of an earlier call.
// Roles (192 threads): warp 0 TMA of B, warp 1 TMEM owner, U2 + MMA issuer, warps 2-5 one thread per token.
constexpr int kFixThreads = 192;
constexpr int kFixCtas = 4;                       // per SM, by their registers
constexpr uint32_t kSmemPerSm = 228 * 1024;       // of which each CTA takes 1 KiB more than it asks for
constexpr uint32_t kFixB = 64 * 128;              // B stage: 64 columns of the output x 64 ranks
constexpr int kFixStages = 16;                    // of B, at most
constexpr uint32_t kFixU = 128 * 128;             // one 64-wide image of U2

constexpr uint32_t kFixSumRow = (64 + 4) * 4;     // a token's sums, padded so that 8 rows' 16 bytes meet no bank twice

struct FixLayout {
    uint32_t off_b, off_sum, off_mask, off_adapter, off_bars, off_slot, off_abort, alloc;
};
__host__ __device__ inline FixLayout fix_layout(uint32_t images, uint32_t tokens, uint32_t stages) {
    FixLayout l;
    l.off_b = images * kFixU;
    l.off_sum = l.off_b + stages * kFixB;
    l.off_mask = l.off_sum + tokens * kFixSumRow;
    l.off_adapter = l.off_mask + 128 * 16;
    l.off_bars = l.off_adapter + 128 * 4;
    l.off_slot = l.off_bars + (2 * kFixStages + 2) * 8;
    l.off_abort = l.off_slot + 4;
    l.alloc = l.off_abort + 4 + 1024;
    return l;
}

// dst[m, 0 .. 64) = the sum of src[b, m, 0 .. 64) over the slots b < n, in order: I chunks of four columns
// a thread and B slots of each in flight.  For a few tokens that spreads a tile's many slots over threads
// that had no token (4 tokens, W[4096, 4096], the whole forward: 21.6 to 20.5 us); for many tokens of few slots
// it is more chunks than slots (112 tokens, W[28672, 8192]: 101.3 to 97.5 us).
template <int I, int B>
__device__ __forceinline__ void sum_slots(const float* src, int64_t slot_floats, int n, int M, int t, char* dst) {
    for (int i0 = t; i0 < M * 16; i0 += 128 * I) {
        float4 acc[I];
#pragma unroll
        for (int i = 0; i < I; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int b0 = 0; b0 < n; b0 += B) {
            float4 v[I][B];
#pragma unroll
            for (int i = 0; i < I; ++i) {
                const int at = i0 + 128 * i;
#pragma unroll
                for (int b = 0; b < B; ++b)
                    v[i][b] = at < M * 16 && b0 + b < n
                                  ? __ldcg(reinterpret_cast<const float4*>(src + (b0 + b) * slot_floats + (at >> 4) * 256) + (at & 15))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < I; ++i)
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    acc[i].x = __fadd_rn(acc[i].x, v[i][b].x);
                    acc[i].y = __fadd_rn(acc[i].y, v[i][b].y);
                    acc[i].z = __fadd_rn(acc[i].z, v[i][b].z);
                    acc[i].w = __fadd_rn(acc[i].w, v[i][b].w);
                }
        }
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int at = i0 + 128 * i;
            if (at < M * 16) reinterpret_cast<float4*>(dst + (at >> 4) * kFixSumRow)[at & 15] = acc[i];
        }
    }
}

__global__ void __launch_bounds__(kFixThreads, kFixCtas)
tc_rows_fixup(const __grid_constant__ CUtensorMap tmU2, const __grid_constant__ CUtensorMap tmB, FixParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - ptx::smem_addr(smem_raw));
    const int images = 2 * p.R / 64;
    const FixLayout lay = fix_layout((uint32_t)images, p.nt, (uint32_t)p.stages);
    const int NS = p.stages;
    const uint32_t sU = base, sB = base + lay.off_b;
    const uint32_t bar_full = base + lay.off_bars, bar_empty = bar_full + 8 * kFixStages;
    const uint32_t bar_u = bar_empty + 8 * kFixStages, bar_acc = bar_u + 8;
    uint32_t* mask = reinterpret_cast<uint32_t*>(gbase + lay.off_mask);       // [adapter place][4]: lanes it leaves alone
    int32_t* adapter = reinterpret_cast<int32_t*>(gbase + lay.off_adapter);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + lay.off_slot);
    volatile int* abort = reinterpret_cast<volatile int*>(gbase + lay.off_abort);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;

    for (int i = tid; i < 128 * 4; i += kFixThreads) mask[i] = 0xffffffffu;
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        ptx::mbar_init(bar_u, 1);
        ptx::mbar_init(bar_acc, 1);
        *abort = 0;
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_smem();
        ptx::tma_prefetch_map(&tmU2);
        ptx::tma_prefetch_map(&tmB);
    }
    if (warp == 1) {
        ptx::tmem_alloc(base + lay.off_slot, 64);
        ptx::tmem_relinquish();
    }
    allow_dependents();
    __syncthreads();
    const int used = __ldcg(p.meta);
    int place = -1;
    if (warp >= 2) {                                          // one thread per token: the lanes of each adapter
        const int m = ((warp & 3) << 5) + lane;
        place = m < p.M ? __ldcg(p.meta + 1 + m) : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, place);
        if (place >= 0 && lane == __ffs((int)same) - 1) {
            mask[place * 4 + (m >> 5)] = ~same;
            adapter[place] = __ldcg(p.idx + m);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int chunks = p.R >= 64 ? p.R / 64 : 1, steps = used * chunks;

    if (warp == 0) {
        int issued = 0, s = 0;
        uint32_t ph = 1;
        for (int i = 0; i < steps; ++i) {
            if (!__all_sync(0xffffffffu, ptx::mbar_wait(bar_empty + 8 * s, ph, abort, p.err))) break;
            issued = i + 1;
            const int d = i / chunks, c = i - d * chunks;
            if (ptx::elect_one_sync()) {
                ptx::mbar_arrive_expect_tx(bar_full + 8 * s, kFixB);
                ptx::tma_load_2d(sB + s * kFixB, &tmB, c * 64, adapter[d] * (int32_t)p.N + (int32_t)blockIdx.x * 64,
                                 bar_full + 8 * s);
            }
            __syncwarp();
            if (++s == NS) { s = 0; ph ^= 1u; }
        }
        if (*abort) {   // drain this CTA's copies in flight before it exits
            for (int i = max(0, issued - NS); i < issued; ++i)
                ptx::mbar_wait_drain(bar_full + 8 * (i % NS), (uint32_t)(i / NS) & 1u);
        }
    } else if (warp == 1) {
        const uint32_t idesc = ptx::idesc_set_f16(ptx::idesc_bf16_f32_ab(128, 64, 0, 0), p.f16 != 0);
        const uint64_t u_sw = ptx::smem_desc_sw128(sU, 16, 1024), b_sw = ptx::smem_desc_sw128(sB, 16, 1024);
        const bool packed = p.R == 32;                        // hi and lo halves of 32 ranks in one image
        grid_dependency_wait();                               // U2 is complete
        if (steps > 0 && ptx::elect_one_sync()) {
            ptx::mbar_arrive_expect_tx(bar_u, (uint32_t)images * kFixU);
            for (int c = 0; c < images; ++c) ptx::tma_load_2d(sU + c * kFixU, &tmU2, c * 64, 0, bar_u);
        }
        __syncwarp();
        bool ok = steps == 0 || __all_sync(0xffffffffu, ptx::mbar_wait(bar_u, 0, abort, p.err));
        int s = 0;
        uint32_t ph = 0;
        for (int i = 0; i < steps && ok; ++i) {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_full + 8 * s, ph, abort, p.err));
            if (!ok) break;
            ptx::tc_fence_after();
            const int d = i / chunks, c = i - d * chunks;
            const uint4 mk = *reinterpret_cast<const uint4*>(mask + d * 4);
            const uint32_t off[4] = {mk.x, mk.y, mk.z, mk.w};
            if (ptx::elect_one_sync()) {
                const uint64_t hi = u_sw + (uint32_t)c * (kFixU >> 4);
                const uint64_t lo = packed ? hi + (64 >> 4) : hi + (uint32_t)chunks * (kFixU >> 4);
                const uint64_t b = b_sw + (uint32_t)s * (kFixB >> 4);
                const int nk = min(4, (p.r - 64 * c + 15) / 16);   // 16-wide steps that hold ranks
                for (int kk = 0; kk < nk; ++kk) {
                    ptx::mma_bf16_ss_lanes(tmem, hi + kk * 2, b + kk * 2, idesc, (c | kk) != 0 ? 1u : 0u, off);
                    ptx::mma_bf16_ss_lanes(tmem, lo + kk * 2, b + kk * 2, idesc, 1u, off);
                }
                ptx::mma_commit(bar_empty + 8 * s);
            }
            __syncwarp();
            if (++s == NS) { s = 0; ph ^= 1u; }
        }
        if (ptx::elect_one_sync()) {
            ptx::mma_commit(bar_acc);
            if (*abort) {   // its copies and issued MMAs finish before the CTA exits and TMEM is freed
                if (steps > 0) ptx::mbar_wait_drain(bar_u, 0);
                ptx::mbar_wait_drain(bar_acc, 0);
            }
        }
        __syncwarp();
    } else {
        const uint32_t quad = (uint32_t)(warp & 3);           // TMEM lanes that the warp reaches: its tokens
        const int m = (int)(quad * 32u) + lane, col0 = (int)(blockIdx.x & 3u) * 64;
        const int per_tile = adapters_per_tile(p.rp), u_tiles = (used + per_tile - 1) / per_tile;
        const int tile = u_tiles + (int)(blockIdx.x >> 2);
        const int2 sp = unit_span((int64_t)tile * p.steps, p.steps, (int64_t)(u_tiles + p.w_tiles) * p.steps, p.G);
        const int slot0 = u_tiles * pieces_of(p.steps) + (tile - u_tiles) + sp.x;
        const bool has = place >= 0;
        const int64_t slot_floats = (int64_t)p.nt * 256;
        const bool live = (int)(quad * 32u) < p.M;
        const float* src = p.partial + (int64_t)slot0 * slot_floats + col0;
        char* sums = reinterpret_cast<char*>(gbase + lay.off_sum);
        const int slots = sp.y - sp.x + 1;
        if (p.M <= 8) sum_slots<1, 12>(src, slot_floats, slots, p.M, tid - 64, sums);
        else if (slots <= 3) sum_slots<6, 3>(src, slot_floats, slots, p.M, tid - 64, sums);
        else sum_slots<4, 6>(src, slot_floats, slots, p.M, tid - 64, sums);
        asm volatile("bar.sync 1, 128;" ::: "memory");        // the sums of other threads
        const bool acc_ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_acc, 0, abort, p.err));
        ptx::tc_fence_after();
        if (acc_ok && live) {
            const int64_t n0 = (int64_t)blockIdx.x * 64;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t v[32];
                ptx::tmem_ld_32x32b_x32(tmem + ((quad * 32u) << 16) + c * 32, v);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (m >= p.M) break;
                    const float4 y = reinterpret_cast<const float4*>(sums + m * kFixSumRow)[8 * c + i];
                    const float x[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[4 * i + e] = __float_as_uint(has ? __fadd_rn(x[e], __uint_as_float(v[4 * i + e])) : x[e]);
                }
                if (m < p.M) store_row32(p.out, p.out_f32 != 0, p.f16 != 0, p.N, m, n0 + 32 * c, p.N, v);
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 64);
    }
}

// ---------------------------------------------------------------------------- host

inline int32_t adapter_rows(int32_t r) { return (r + 7) / 8 * 8; }

inline uint32_t token_tile(int64_t M) { return (uint32_t)((M + 7) / 8 * 8); }

}  // namespace

// Pieces of A_all rows that M tokens can use.
static int64_t u_pieces(int64_t M, int64_t K, int32_t r, int64_t n_adapters) {
    const int64_t per_tile = adapters_per_tile(adapter_rows(r));
    return (std::min(M, n_adapters) + per_tile - 1) / per_tile * pieces_of((int)(K / 64));
}

// meta [1 + 128] int32 in 1 KiB, the pieces' CTAs, then the partial tiles: one slot for each piece and W
// tile and one for each CTA boundary.
size_t rows_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t r, int64_t n_adapters) {
    const int64_t pieces = u_pieces(M, K, r, n_adapters), slots = (N + 255) / 256 + pieces + kMaxCtas;
    return 1024 + align_up((size_t)pieces * 8, 256) + (size_t)slots * token_tile(M) * 256 * sizeof(float);
}

qlora_status launch_rows(const RowsArgs& a, cudaStream_t stream) {
    const qlora_nf4_weight* w = a.w;
    const int64_t N = w->N, K = w->K;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return QLORA_ERR_CUDA;
    static std::atomic<uint64_t> configured{0}, fix_configured{0};
    if (!allow_smem(configured, (const void*)tc_rows_nf4, (int)kMaxSmem) ||
        !allow_smem(fix_configured, (const void*)tc_rows_fixup, (int)kMaxSmem))
        return QLORA_ERR_CUDA;
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
    p.piece_ctas = reinterpret_cast<int2*>(static_cast<char*>(a.workspace) + 1024);
    p.partial = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + 1024 +
                                         align_up((size_t)u_pieces(a.M, K, a.r, a.n_adapters) * 8, 256));
    p.tb = host_tables(w->codebook);
    p.err = device_error_word();
    if (!p.err) return QLORA_ERR_CUDA;
    CUtensorMap tmCodes, tmX, tmA;
    if (!make_tmap_codes32(&tmCodes, w->codes, K / 2, N)) return QLORA_ERR_CUDA;
    if (!make_tmap_3d(&tmA, a.A, K, a.r, a.n_adapters, 64, (uint32_t)p.rp)) return QLORA_ERR_CUDA;
    if (!make_tmap_2d(&tmX, true, a.X, K, a.M, K * 2, 64, p.nt, true)) return QLORA_ERR_CUDA;
    // At least sqrt(K / 64) / 2 units per CTA: a unit costs its CTA about what a further slot costs the
    // fix-up, and a tile's slots are its K / 64 units over a CTA's number of them (W[1024, 1024]: 33 to
    // 31 us at 100 tokens).
    int64_t least = 1;
    while (4 * least * least < p.steps) ++least;
    const int64_t G = std::max<int64_t>(1, std::min<int64_t>({(int64_t)p.w_tiles * p.steps / least, (int64_t)sms, (int64_t)kMaxCtas}));
    (void)launch_dependent(tc_rows_nf4, dim3((unsigned)G), dim3(kThreads), lay.alloc, stream, tmCodes, tmX, tmA, p);
    QLORA_CHECK_LAUNCH();
    FixParams f{};
    f.partial = p.partial; f.piece_ctas = p.piece_ctas; f.meta = p.meta; f.idx = a.idx; f.scales = a.scales; f.U = a.U; f.out = a.out; f.N = N;
    f.U2 = static_cast<uint16_t*>(a.U2);
    f.M = p.M; f.r = p.r; f.R = a.R; f.rp = p.rp; f.steps = p.steps; f.w_tiles = p.w_tiles; f.G = (int32_t)G;
    f.all_pieces = (int32_t)u_pieces(a.M, K, a.r, a.n_adapters);
    f.nt = p.nt; f.out_f32 = a.out_f32; f.f16 = p.f16; f.err = p.err;
    (void)launch_dependent(rows_finish_U, dim3((unsigned)((f.M * f.R + 127) / 128)), dim3(128), 0, stream, f);
    QLORA_CHECK_LAUNCH();
    CUtensorMap tmU2, tmB;
    if (!make_tmap_2d(&tmU2, true, a.U2, 2 * a.R, a.M, 4 * a.R, 64, 128, true)) return QLORA_ERR_CUDA;
    if (!make_tmap_2d(&tmB, true, a.B, a.ldb, (uint64_t)a.n_adapters * N, a.ldb * 2, 64, 64, true)) return QLORA_ERR_CUDA;
    // As many stages of B as a CTA can use (an adapter's tile takes one for every 64 ranks) and as let all CTAs
    // run together, at least two; four if no number does (48 tokens, 32 adapters, the whole forward: W[28672, 8192],
    // 448 CTAs, 105.5 us with four stages and 102 with two; W[8192, 8192] 47.9 with four and 47.4 with sixteen).
    const int64_t ctas = (N + 63) / 64, tiles = std::min<int64_t>(a.M, a.n_adapters) * ((a.r + 63) / 64);
    const uint32_t images = (uint32_t)(2 * a.R / 64);
    f.stages = 4;
    for (int st = (int)std::min<int64_t>(kFixStages, std::max<int64_t>(2, tiles)); st >= 2; --st) {
        const uint32_t bytes = fix_layout(images, f.nt, (uint32_t)st).alloc;
        if (bytes <= kMaxSmem && std::min<int64_t>(kFixCtas, kSmemPerSm / (bytes + 1024)) * sms >= ctas) {
            f.stages = st;
            break;
        }
    }
    (void)launch_dependent(tc_rows_fixup, dim3((unsigned)ctas), dim3(kFixThreads),
                           fix_layout(images, f.nt, (uint32_t)f.stages).alloc, stream, tmU2, tmB, f);
    QLORA_CHECK_LAUNCH();
    return QLORA_OK;
}

}  // namespace qlora
