// Forward of up to 128 tokens, each with its own adapter, over one quantized weight: the decode step
// of many requests (one token each, drafted tokens, or short prompts).
//
//     Y[m] = X[m] W_hat^T + s_a (X[m] A_a^T) B_a^T,   a = adapter_idx[m]
//
// The products with the long reduction over K run in one persistent kernel, "swap-AB": D[row, token]
// with 128 rows as the MMA's M and the tokens, rounded up to 16, as its N.  The rows are first those of
// A_all of the adapters that the batch uses (found by every CTA from the M indices; each adapter takes
// its rank rounded up to a power of two), then those of W_hat.  An adapter's rows meet every token and
// only the products with its own are read, which costs tensor-core time that is idle here, and no token
// meets another's adapter in a sum.
//
// Work units are 128 rows x 128 of K; the units, tile major, are cut into equal contiguous ranges, one
// per CTA (one CTA per SM), and every (tile, CTA) piece is a segment accumulated in TMEM and written as
// an fp32 partial tile to slot tile + CTA.  rows_fixup sums each tile's slots in CTA order, adds the
// adapter term s_a U B_a^T in fp32 and writes Y.
//
// The expansion of the codes bounds the kernel (byte permutes, two to three ALU operations a weight),
// so a unit holds two blocks of 64 weights per thread, twice the 64-wide unit of tc_decode_nf4, which
// halves the handshakes per weight, and the producer warps of one CTA share its rings.
// Roles: warp 0 TMA, warp 1 TMEM owner + MMA issuer, then four groups of four producer warps (three
// when the token tile leaves no room for four) that take units in turn, and segments' epilogues in turn.
//
// A parity wait tells apart only neighbouring phases, so no role may come to a barrier two phases
// behind.  Producers skip other groups' units; what they have seen suffices because the row ring has at
// least as many stages as there are groups, the token ring at least as many as the row ring, each unit's
// row stage is waited for before its tokens, and every group has an accumulator of its own.
#include <algorithm>
#include <climits>

#include "gemm_tc.cuh"
#include "nf4_expand.cuh"
#include "qlora_internal.cuh"
#include "tc_ptx.cuh"

namespace qlora {
namespace {

constexpr int kMaxGroups = 4;
constexpr int kMaxCtas = 256;
constexpr uint32_t kAStage = 128 * 256;           // 128 rows x 128 16-bit elements
constexpr uint32_t kCodes = 128 * 64;             // their packed codes
constexpr uint32_t kMaxSmem = 227 * 1024;
constexpr int kPrefetch = 2;                      // block constants are loaded this many units (of the group) ahead

struct RowsLayout {
    uint32_t c_stage, off_c, off_ids, off_list, off_bars, off_slot, off_abort, alloc;
};
__host__ __device__ inline RowsLayout rows_layout(uint32_t nt, uint32_t as, uint32_t cs) {
    RowsLayout l;
    l.c_stage = kCodes + nt * 256u;               // X as two [nt x 64] swizzled images, then the codes
    l.off_c = as * kAStage;
    l.off_ids = l.off_c + cs * l.c_stage;         // adapter of each token [128]
    l.off_list = l.off_ids + 128 * 4;             // adapters that the batch uses [128]
    l.off_bars = l.off_list + 128 * 4;
    l.off_slot = l.off_bars + (2 * as + 2 * cs + 2 * kMaxGroups + 1) * 8;
    l.off_abort = l.off_slot + 4;
    l.alloc = l.off_abort + 4 + 16 + 1024;        // + ballots [4]
    return l;
}

struct RowsParams {
    int32_t M, r, rp;                             // rp: rows an adapter takes (a power of two of at least 16)
    int32_t steps;                                // units per tile
    int32_t w_tiles;                              // tiles of W_hat rows
    int64_t N, K;
    const int32_t* idx;
    int32_t n_adapters;
    const uint8_t* c1_codes;
    const float* c2;
    const float* mu;
    const float* c1f;
    int32_t f16;
    uint32_t nt, a_stages, c_stages, tmem_cols;
    float* partial;                               // [tiles + CTAs][nt][128]
    int32_t* meta;                                // [0] adapters in use, [1 + m] place of token m's adapter among them, or -1
    uint32_t* err;
    NF4Tables tb;
};

__host__ __device__ __forceinline__ int64_t range_begin(int64_t b, int64_t units, int64_t G) { return b * units / G; }

template <int GROUPS>
__global__ void __launch_bounds__(64 + 128 * GROUPS, 1)
tc_rows_nf4(const __grid_constant__ CUtensorMap tmCodes, const __grid_constant__ CUtensorMap tmX,
            const __grid_constant__ CUtensorMap tmA, RowsParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - ptx::smem_addr(smem_raw));
    const int AS = (int)p.a_stages, CS = (int)p.c_stages;
    const RowsLayout lay = rows_layout(p.nt, p.a_stages, p.c_stages);
    const uint32_t sA = base, sC = base + lay.off_c, xbytes = p.nt * 256u;
    int32_t* ids = reinterpret_cast<int32_t*>(gbase + lay.off_ids);
    int32_t* list = reinterpret_cast<int32_t*>(gbase + lay.off_list);
    const uint32_t bar_cfull = base + lay.off_bars, bar_cempty = bar_cfull + 8 * CS;
    const uint32_t bar_afull = bar_cempty + 8 * CS, bar_aempty = bar_afull + 8 * AS;
    const uint32_t bar_accfull = bar_aempty + 8 * AS, bar_accempty = bar_accfull + 8 * GROUPS, bar_drain = bar_accempty + 8 * GROUPS;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + lay.off_slot);
    volatile int* abort = reinterpret_cast<volatile int*>(gbase + lay.off_abort);
    volatile uint32_t* ballots = reinterpret_cast<volatile uint32_t*>(gbase + lay.off_abort + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;

    allow_dependents();
    if (tid == 0) {
        for (int s = 0; s < CS; ++s) {
            ptx::mbar_init(bar_cfull + 8 * s, 1);
            ptx::mbar_init(bar_cempty + 8 * s, 1);
        }
        for (int s = 0; s < AS; ++s) {
            ptx::mbar_init(bar_afull + 8 * s, 4);
            ptx::mbar_init(bar_aempty + 8 * s, 1);
        }
        for (int a = 0; a < GROUPS; ++a) {
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
        ptx::tmem_alloc(base + lay.off_slot, p.tmem_cols);
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
        for (int j = tid - 1; j >= 0; --j)
            if (ids[j] == a) first = j;
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
    const int u_tiles = (used * p.rp + 127) / 128;            // tiles of A_all rows come first
    const int64_t units = (int64_t)(u_tiles + p.w_tiles) * S;
    const int64_t u0 = range_begin(blockIdx.x, units, gridDim.x);
    const int n = (int)(range_begin(blockIdx.x + 1, units, gridDim.x) - u0);
    const int t0 = (int)(u0 / S), step0 = (int)(u0 - (int64_t)t0 * S);

    if (warp == 0) {
        // unit i: X (and the codes, or the adapters' rows) into ring slot i % CS once the MMA that read the
        // slot before has completed
        bool ok = true;
        int issued = 0, tile = t0, step = step0, cs = 0, s = 0;
        uint32_t cph = 0, ph = 0;
        const int per_tile = p.rp >= 128 ? 1 : 128 / p.rp;    // adapters in a tile of A_all rows
        const uint32_t box_bytes = (uint32_t)min(p.rp, 128) * 128u;
        for (int i = 0; i < n && ok; ++i) {
            const bool is_u = tile < u_tiles;
            bool w = ptx::mbar_wait(bar_cempty + 8 * cs, cph ^ 1u, abort, p.err);
            if (w && is_u) w = ptx::mbar_wait(bar_aempty + 8 * s, ph ^ 1u, abort, p.err);
            ok = __all_sync(0xffffffffu, w);
            if (!ok) break;
            if (ptx::elect_one_sync()) {
                const uint32_t fb = bar_cfull + 8 * cs, x = sC + cs * lay.c_stage;
                const int u_row = tile * 128;
                const int ad0 = u_row / p.rp, ads = is_u ? min(per_tile, used - ad0) : 0;
                ptx::mbar_arrive_expect_tx(fb, xbytes + (is_u ? 2u * box_bytes * (uint32_t)ads : kCodes));
                ptx::tma_load_2d(x, &tmX, step * 128, 0, fb);
                ptx::tma_load_2d(x + p.nt * 128u, &tmX, step * 128 + 64, 0, fb);
                if (!is_u) {
                    ptx::tma_load_2d(x + xbytes, &tmCodes, step * 64, (tile - u_tiles) * 128, fb);
                } else {
                    for (int q = 0; q < ads; ++q) {
                        const uint32_t dst = sA + s * kAStage + (uint32_t)q * box_bytes;
                        const int rank0 = u_row - (ad0 + q) * p.rp > 0 ? u_row - (ad0 + q) * p.rp : 0;
                        ptx::tma_load_3d(dst, &tmA, step * 128, rank0, list[ad0 + q], fb);
                        ptx::tma_load_3d(dst + 16384, &tmA, step * 128 + 64, rank0, list[ad0 + q], fb);
                    }
                }
            }
            __syncwarp();
            issued = i + 1;
            if (++step == S) { step = 0; ++tile; }
            if (++cs == CS) { cs = 0; cph ^= 1u; }
            if (++s == AS) { s = 0; ph ^= 1u; }
        }
        if (*abort) {   // drain this CTA's copies in flight before it exits
            for (int c = max(0, issued - CS); c < issued; ++c)
                ptx::mbar_wait_drain(bar_cfull + 8 * (c % CS), (uint32_t)(c / CS) & 1u);
        }
    } else if (warp == 1) {
        const uint32_t idesc = ptx::idesc_set_f16(ptx::idesc_bf16_f32_ab(128, (int)p.nt, 0, 0), p.f16 != 0);
        const uint64_t a_none = ptx::smem_desc_kmajor_none(sA, 128 * 16, 128);   // W_hat rows, as the producers write them
        const uint64_t a_sw = ptx::smem_desc_sw128(sA, 16, 1024);                // A_all rows, as TMA does
        const uint64_t x_sw = ptx::smem_desc_sw128(sC, 16, 1024);
        bool ok = true, fresh = true;
        int tile = t0, step = step0, acc = 0, s = 0, cs = 0;
        uint32_t ph = 0, cph = 0, acc_ph = 1;                 // accumulator of the segment at hand and its use, mod 2
        for (int i = 0; i < n && ok; ++i) {
            if (fresh) {                                      // drained by the epilogue of its last segment
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_accempty + 8 * acc, acc_ph, abort, p.err));
                if (!ok) break;
            }
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_afull + 8 * s, ph, abort, p.err) &&
                                             ptx::mbar_wait(bar_cfull + 8 * cs, cph, abort, p.err));
            if (!ok) break;
            ptx::tc_fence_after();
            const bool last = (step + 1 == S) || (i == n - 1);
            if (ptx::elect_one_sync()) {
                const bool is_u = tile < u_tiles;
                const uint64_t ad = (is_u ? a_sw : a_none) + ((uint32_t)s * (kAStage >> 4));
                const uint64_t bd = x_sw + ((uint32_t)cs * (lay.c_stage >> 4));
                const uint32_t d = tmem + p.nt * (uint32_t)acc;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint32_t ak = is_u ? (kk >> 2) * (16384u >> 4) + (kk & 3) * (32u >> 4) : kk * ((2u * 128 * 16) >> 4);
                    const uint32_t bk = (kk >> 2) * ((p.nt * 128u) >> 4) + (kk & 3) * (32u >> 4);
                    ptx::mma_bf16_ss(d, ad + ak, bd + bk, idesc, (fresh && kk == 0) ? 0u : 1u);
                }
                ptx::mma_commit(bar_aempty + 8 * s);
                ptx::mma_commit(bar_cempty + 8 * cs);
                if (last) ptx::mma_commit(bar_accfull + 8 * acc);   // the segment ends: hand the accumulator over
            }
            __syncwarp();
            if (++s == AS) { s = 0; ph ^= 1u; }
            if (++cs == CS) { cs = 0; cph ^= 1u; }
            fresh = last;
            if (++step == S) { step = 0; ++tile; }
            if (last && ++acc == GROUPS) { acc = 0; acc_ph ^= 1u; }
        }
        if (ptx::elect_one_sync()) {
            ptx::mma_commit(bar_drain);
            if (*abort) ptx::mbar_wait_drain(bar_drain, 0);   // issued MMAs finish before TMEM is freed
        }
        __syncwarp();
    } else {
        // group g takes units g, g + GROUPS, ...; thread t expands row t of the unit's tile, two blocks of 64
        const int g = (warp - 2) >> 2, t = tid - 64 - 128 * g;
        const int kb = (int)(p.K / 64);
        const float mu = p.c1f ? 0.f : *p.mu;
        const int32_t wrow0 = t - u_tiles * 128;              // W row of thread t in tile 0
        struct Cursor { int tile, step; };
        auto advance = [&](Cursor& c, int by) {
            c.step += by;
            while (c.step >= S) { c.step -= S; ++c.tile; }
        };
        // block constants of a unit: the E4M3 codes (or fp32 constants) of its two blocks and their c2
        struct Consts { uint32_t code; float c2a, c2b; };
        auto load_consts = [&](const Cursor& c) {
            Consts k{0, 0.f, 0.f};
            const int64_t row = (int64_t)wrow0 + (int64_t)c.tile * 128;
            if (c.tile < u_tiles || row >= p.N) return k;
            const int b0 = 2 * c.step;
            const int64_t blk = row * kb + b0;
            const bool two = b0 + 1 < kb;
            if (p.c1f) {
                k.c2a = __ldg(p.c1f + blk);
                if (two) k.c2b = __ldg(p.c1f + blk + 1);
            } else {
                k.code = __ldg(p.c1_codes + blk);
                k.c2a = __ldg(p.c2 + (blk >> 8));
                if (two) {
                    k.code |= (uint32_t)__ldg(p.c1_codes + blk + 1) << 8;
                    k.c2b = __ldg(p.c2 + ((blk + 1) >> 8));
                }
            }
            return k;
        };
        Cursor cur{t0, step0};
        advance(cur, g);
        Cursor pf = cur;
        Consts q[kPrefetch];
#pragma unroll
        for (int d = 0; d < kPrefetch; ++d) {
            q[d] = Consts{0, 0.f, 0.f};
            if (g + GROUPS * d < n) q[d] = load_consts(pf);
            advance(pf, GROUPS);
        }

        int epi_seg = g;                                      // next segment whose epilogue is this group's
        const int last_seg = (int)((u0 + n - 1) / S) - t0;
        auto epilogue = [&](int seg) -> bool {
            const bool ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_accfull + 8 * g, (uint32_t)(seg / GROUPS) & 1u,
                                                                    abort, p.err));
            if (!ok) return false;
            ptx::tc_fence_after();
            const uint32_t quad = (uint32_t)(warp & 3);
            float* dst = p.partial + (int64_t)(t0 + seg + blockIdx.x) * p.nt * 128 + quad * 32 + lane;
#pragma unroll 1
            for (uint32_t c = 0; c < p.nt; c += 16) {
                uint32_t v[16];
                ptx::tmem_ld_32x32b_x16(tmem + ((quad * 32u) << 16) + p.nt * (uint32_t)g + c, v);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int m = 0; m < 16; ++m)
                    if ((int)c + m < p.M) dst[(c + m) * 128] = __uint_as_float(v[m]);
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_accempty + 8 * g);
            return true;
        };

        bool ok = true;
        int cs = g % CS, s = g % AS;
        uint32_t cph = (uint32_t)(g / CS) & 1u, ph = (uint32_t)(g / AS) & 1u;
        for (int i = g; i < n && ok; i += GROUPS) {
            const int seg = cur.tile - t0;
            while (epi_seg < seg && ok) { ok = epilogue(epi_seg); epi_seg += GROUPS; }
            if (!ok) break;
            const Consts k = q[0];
#pragma unroll
            for (int d = 0; d + 1 < kPrefetch; ++d) q[d] = q[d + 1];
            q[kPrefetch - 1] = Consts{0, 0.f, 0.f};
            if (i + GROUPS * kPrefetch < n) q[kPrefetch - 1] = load_consts(pf);
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_aempty + 8 * s, ph ^ 1u, abort, p.err) &&
                                             ptx::mbar_wait(bar_cfull + 8 * cs, cph, abort, p.err));
            if (!ok) break;
            if (cur.tile >= u_tiles) {
                const bool row_ok = (int64_t)wrow0 + (int64_t)cur.tile * 128 < p.N;
                const bool two = row_ok && 2 * cur.step + 1 < kb;
                const uint32_t row_addr = sA + s * kAStage + (uint32_t)t * 16u;
                const uint32_t src = sC + cs * lay.c_stage + xbytes + (uint32_t)t * 64u, swz = ((uint32_t)t >> 1) & 3u;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint32_t dst = row_addr + b * 8u * 2048u;
                    if (!(b == 0 ? row_ok : two)) {
                        zero_row_kn<2048>(dst);
                        continue;
                    }
                    const uint4 x = ld_shared_v4(src + (((2u * b) ^ swz) << 4));
                    const uint4 y = ld_shared_v4(src + (((2u * b + 1u) ^ swz) << 4));
                    const float c2 = b ? k.c2b : k.c2a;
                    const float c1p = p.c1f ? c2 : __fadd_rn(__fmul_rn(e4m3_to_f32((k.code >> (8 * b)) & 255u), c2), mu);
                    Lut lut;
                    build_lut(lut, c1p, p.tb, p.f16 != 0);
                    expand_block_row_kn<2048>(dst, x, y, lut);
                }
                ptx::fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_afull + 8 * s);
            advance(cur, GROUPS);
            advance(pf, GROUPS);
            cs += GROUPS;
            while (cs >= CS) { cs -= CS; cph ^= 1u; }
            s += GROUPS;
            while (s >= AS) { s -= AS; ph ^= 1u; }
        }
        while (ok && epi_seg <= last_seg) { ok = epilogue(epi_seg); epi_seg += GROUPS; }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, p.tmem_cols);
    }
}

// Y[m, n] = the sum of the partial tiles of n / 128 in CTA order + s_a sum_j U[m, j] B_a[n, j] (ascending
// j, fp32), rounded to the output type.  CTA (tile, y): 128 rows of W, tokens 16 y .. 16 y + 15.  U is
// summed from its own partial tiles first; the CTAs of tile 0 also store it.
constexpr int kFixTokens = 16;

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

__global__ void __launch_bounds__(128)
rows_fixup(FixParams p) {
    extern __shared__ float us[];                             // us[q * (r + 4) + j] = U[m0 + q, j]
    __shared__ int32_t tok_place[kFixTokens], tok_adapter[kFixTokens];
    const int tid = threadIdx.x, m0 = (int)blockIdx.y * kFixTokens, nm = min(p.M - m0, kFixTokens);
    grid_dependency_wait();                                   // partial tiles are complete
    if (tid < kFixTokens) {
        const int place = tid < nm ? p.meta[1 + m0 + tid] : -1;
        tok_place[tid] = place;
        tok_adapter[tid] = place >= 0 ? p.idx[m0 + tid] : -1;
    }
    const int u_tiles = (p.meta[0] * p.rp + 127) / 128;
    const int64_t units = (int64_t)(u_tiles + p.w_tiles) * p.steps;
    const int64_t slot_floats = (int64_t)p.nt * 128;
    auto cta_of = [&](int64_t u) {                            // the CTA whose range holds unit u
        int64_t b = u * p.G / units;
        while (b + 1 < p.G && range_begin(b + 1, units, p.G) <= u) ++b;
        while (b > 0 && range_begin(b, units, p.G) > u) --b;
        return (int)b;
    };
    __syncthreads();
    const int pitch = p.r + 4;                                // keeps rows 16-byte aligned for r % 4 == 0
    for (int i = tid; i < kFixTokens * p.r; i += 128) {
        const int q = i / p.r, j = i - q * p.r;
        float v = 0.f;
        if (tok_place[q] >= 0) {
            const int row = tok_place[q] * p.rp + j, tile = row >> 7;
            const int ba = cta_of((int64_t)tile * p.steps), bz = cta_of((int64_t)tile * p.steps + p.steps - 1);
            const float* src = p.partial + (int64_t)tile * slot_floats + (int64_t)(m0 + q) * 128 + (row & 127);
            for (int b = ba; b <= bz; ++b) v = __fadd_rn(v, src[(int64_t)b * slot_floats]);
        }
        us[q * pitch + j] = v;
        if (p.U && blockIdx.x == 0 && q < nm) p.U[(int64_t)(m0 + q) * p.r + j] = v;
    }
    __syncthreads();
    const int tile = u_tiles + (int)blockIdx.x;
    const int64_t n = (int64_t)blockIdx.x * 128 + tid;
    if (n >= p.N) return;
    float lora[kFixTokens];
#pragma unroll
    for (int q = 0; q < kFixTokens; ++q) lora[q] = 0.f;
    const bool f16 = p.f16 != 0;
    for (int j0 = 0; j0 < p.r; j0 += 8) {
        float bv[8];
        int have = -1;
#pragma unroll
        for (int q = 0; q < kFixTokens; ++q) {
            const int a = tok_adapter[q];
            if (a < 0) continue;
            if (a != have) {                                  // tokens of one request follow each other
                have = a;
                const uint16_t* br = p.B + ((int64_t)a * p.N + n) * p.r + j0;
                if ((p.r & 7) == 0) {
                    const uint4 w = __ldg(reinterpret_cast<const uint4*>(br));
                    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        bv[2 * e] = from16(v[e] & 0xFFFFu, f16);
                        bv[2 * e + 1] = from16(v[e] >> 16, f16);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) bv[e] = j0 + e < p.r ? from16(br[e], f16) : 0.f;
                }
            }
            if ((p.r & 7) == 0) {
                const float4 u0 = *reinterpret_cast<const float4*>(us + q * pitch + j0);
                const float4 u1 = *reinterpret_cast<const float4*>(us + q * pitch + j0 + 4);
                lora[q] = __fmaf_rn(u0.x, bv[0], lora[q]);
                lora[q] = __fmaf_rn(u0.y, bv[1], lora[q]);
                lora[q] = __fmaf_rn(u0.z, bv[2], lora[q]);
                lora[q] = __fmaf_rn(u0.w, bv[3], lora[q]);
                lora[q] = __fmaf_rn(u1.x, bv[4], lora[q]);
                lora[q] = __fmaf_rn(u1.y, bv[5], lora[q]);
                lora[q] = __fmaf_rn(u1.z, bv[6], lora[q]);
                lora[q] = __fmaf_rn(u1.w, bv[7], lora[q]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (j0 + e < p.r) lora[q] = __fmaf_rn(us[q * pitch + j0 + e], bv[e], lora[q]);
            }
        }
    }
    const int ba = cta_of((int64_t)tile * p.steps), bz = cta_of((int64_t)tile * p.steps + p.steps - 1);
    float acc[kFixTokens];
#pragma unroll
    for (int q = 0; q < kFixTokens; ++q) acc[q] = 0.f;
    for (int b = ba; b <= bz; ++b) {
        const float* src = p.partial + (int64_t)(tile + b) * slot_floats + (int64_t)m0 * 128 + tid;
        float v[kFixTokens];
#pragma unroll
        for (int q = 0; q < kFixTokens; ++q) v[q] = q < nm ? src[q * 128] : 0.f;
#pragma unroll
        for (int q = 0; q < kFixTokens; ++q) acc[q] = __fadd_rn(acc[q], v[q]);
    }
#pragma unroll
    for (int q = 0; q < kFixTokens; ++q) {
        if (q >= nm) break;
        const int a = tok_adapter[q];
        const float y = a >= 0 ? __fmaf_rn(__ldg(p.scales + a), lora[q], acc[q]) : acc[q];
        const int64_t at = (int64_t)(m0 + q) * p.N + n;
        if (p.out_f32) static_cast<float*>(p.out)[at] = y;
        else static_cast<uint16_t*>(p.out)[at] = (uint16_t)to16_rn(y, f16);
    }
}

// ---------------------------------------------------------------------------- host

int32_t adapter_rows(int32_t r) {
    int32_t rp = 16;
    while (rp < r) rp *= 2;
    return rp;
}

template <int GROUPS>
qlora_status launch_units(int64_t G, uint32_t smem, cudaStream_t s, const CUtensorMap& tmCodes, const CUtensorMap& tmX,
                          const CUtensorMap& tmA, const RowsParams& p) {
    static bool configured = false;   // attribute set once per instantiation (idempotent, so races are benign)
    auto kern = tc_rows_nf4<GROUPS>;
    if (!configured) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem) != cudaSuccess)
            return QLORA_ERR_CUDA;
        configured = true;
    }
    (void)launch_dependent(kern, dim3((unsigned)G), dim3(64 + 128 * GROUPS), smem, s, tmCodes, tmX, tmA, p);
    QLORA_CHECK_LAUNCH();
    return QLORA_OK;
}

inline uint32_t token_tile(int64_t M) { return (uint32_t)((M + 15) / 16 * 16); }

}  // namespace

// meta [1 + 128] int32, then the partial tiles of every W tile and of the tiles of A_all rows that M
// tokens can use, plus one for each CTA boundary.
size_t rows_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t r, int64_t n_adapters) {
    const int64_t tiles = (N + 127) / 128 + (std::min(M, n_adapters) * adapter_rows(r) + 127) / 128;
    return 1024 + (size_t)(tiles + kMaxCtas) * token_tile(M) * 128 * sizeof(float);
}

qlora_status launch_rows(const RowsArgs& a, cudaStream_t stream) {
    const qlora_nf4_weight* w = a.w;
    const int64_t N = w->N, K = w->K;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return QLORA_ERR_CUDA;
    RowsParams p{};
    p.M = (int32_t)a.M; p.r = a.r; p.rp = adapter_rows(a.r);
    p.steps = (int32_t)((K + 127) / 128);
    p.w_tiles = (int32_t)((N + 127) / 128);
    p.N = N; p.K = K;
    p.idx = a.idx; p.n_adapters = a.n_adapters;
    p.c1_codes = w->c1_codes; p.c2 = w->c2; p.mu = w->mu; p.c1f = w->c1;
    p.f16 = w->compute_dtype == QLORA_DTYPE_F16;
    p.nt = token_tile(a.M);
    // Groups of producers = row stages = accumulators, and at least as many token stages: four where
    // they fit (up to 64 tokens), else three.  More token stages where there is room, at most two for
    // each row stage.
    int groups = kMaxGroups;
    if (rows_layout(p.nt, 4, 4).alloc > kMaxSmem) groups = 3;
    p.a_stages = (uint32_t)groups;
    p.c_stages = 2 * p.a_stages;
    while (p.c_stages > p.a_stages && rows_layout(p.nt, p.a_stages, p.c_stages).alloc > kMaxSmem) --p.c_stages;
    const RowsLayout lay = rows_layout(p.nt, p.a_stages, p.c_stages);
    if (lay.alloc > kMaxSmem) return QLORA_ERR_UNSUPPORTED;
    p.tmem_cols = 32;
    while (p.tmem_cols < (uint32_t)groups * p.nt) p.tmem_cols *= 2;
    p.meta = static_cast<int32_t*>(a.workspace);
    p.partial = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + 1024);
    p.tb = host_tables(w->codebook);
    p.err = device_error_word();
    if (!p.err) return QLORA_ERR_CUDA;
    CUtensorMap tmCodes, tmX, tmA;
    if (!make_tmap_codes64(&tmCodes, w->codes, K / 2, N)) return QLORA_ERR_CUDA;
    if (!make_tmap_2d(&tmX, true, a.X, K, a.M, K * 2, 64, p.nt, true)) return QLORA_ERR_CUDA;
    if (!make_tmap_3d(&tmA, a.A, K, a.r, a.n_adapters, 64, (uint32_t)std::min(p.rp, 128))) return QLORA_ERR_CUDA;
    const int64_t G = std::min<int64_t>({(int64_t)p.w_tiles * p.steps, (int64_t)sms, (int64_t)kMaxCtas});
    QLORA_TRY(groups == 4 ? launch_units<4>(G, lay.alloc, stream, tmCodes, tmX, tmA, p)
                          : launch_units<3>(G, lay.alloc, stream, tmCodes, tmX, tmA, p));
    FixParams f{};
    f.partial = p.partial; f.meta = p.meta; f.idx = a.idx; f.scales = a.scales;
    f.B = static_cast<const uint16_t*>(a.B); f.U = a.U; f.out = a.out; f.N = N;
    f.M = p.M; f.r = p.r; f.rp = p.rp; f.steps = p.steps; f.w_tiles = p.w_tiles; f.G = (int32_t)G; f.nt = p.nt;
    f.out_f32 = a.out_f32; f.f16 = p.f16;
    const dim3 grid((unsigned)p.w_tiles, (unsigned)((a.M + kFixTokens - 1) / kFixTokens));
    (void)launch_dependent(rows_fixup, grid, dim3(128), (size_t)(a.r + 4) * kFixTokens * sizeof(float), stream, f);
    QLORA_CHECK_LAUNCH();
    return QLORA_OK;
}

}  // namespace qlora
