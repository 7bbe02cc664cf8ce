// The linear layer with one adapter per token: the low-rank adapters of many requests at once
// beside the shared quantized projection, forward and backward ("Ch.09 QLoRA 与量化", section
// "3. 一个底座，多个适配器": one shared compressed base, one thin adapter per task).
//
// With a = adapter_idx[m] (none: a = -1) and s_a = scales[a]:
//     U[m]  = X[m] A_a^T                     Y[m]  = X[m] W_hat^T + s_a U[m] B_a^T
//     dU[m] = s_a dY[m] B_a                  dX[m] = dY[m] W_hat + dU[m] A_a
//     dA_a  = sum over its tokens of dU[m]^T X[m]
//     dB_a  = sum over its tokens of s_a dY[m]^T U[m]
//
// Tokens stay where they are: nothing is sorted or gathered.  Lists built on the device say which
// adapters occur in which token tile and in which of its rows, and
//   - products whose rows are tokens (U, dU here; Y and dX in gemm_tc.cu) run one pass per adapter of
//     the tile, whose MMAs write only that adapter's rows (the output-lane mask of tcgen05.mma);
//   - products that sum over tokens (dA, dB) run over the adapter's own token tiles, and a tile that
//     it shares has the other tokens' rows zeroed in shared memory first, so that Inf or NaN in one
//     request's activations stays out of another's gradient.
// A tile of contiguous requests meets few adapters, so the passes cost little; any order of tokens is
// correct.
#include <climits>
#include <algorithm>

#include "gemm_tc.cuh"
#include "qlora_internal.cuh"
#include "tc_ptx.cuh"
#include "timing.cuh"

namespace qlora {
namespace {

constexpr int kPartTile = 128;                    // token rows of a U / dU tile
constexpr int kGradTile = 64;                     // tokens of one reduction step of dA / dB
constexpr uint32_t kStage16K = 128 * 128;
constexpr uint32_t kMaxSmem = 227 * 1024;

// ---------------------------------------------------------------------------- lists

// What the kernels below read of adapter_idx; all pieces live in the caller's workspace.
struct AdapterLists {
    int32_t* tok;             // [M] adapter of each token, -1 for none or an index out of range
    uint32_t* n512;           // [tiles of 512] entries of the tile
    uint32_t* e512;           // [tiles of 512][cap512][kAdEntry]
    uint32_t* n_grad;         // [n_adapters] token tiles of 64 that hold the adapter
    uint4* e_grad;            // [n_adapters][tiles of 64]: tile, row mask (2 words), 1 if no other rows
    int32_t cap512;
    int32_t tiles64;
};

// Block b < tiles512: the list of tokens 512 b .. 512 b + 511, one thread per token.  The first token of
// the tile with an adapter opens its entry (entries in order of first appearance, so the lists do not
// depend on timing), and each warp's tokens of one adapter write one word of its mask.  The first token
// comes from a minimum per adapter in shared memory (up to 8192 adapters; a search of the tile above).
// Block tiles512 + a: the token tiles of adapter a.
constexpr int kTableAdapters = 8192;
constexpr int kGradBatch = 4;                     // 512-token pieces whose indices are loaded together

__global__ void __launch_bounds__(512)
build_lists(const int32_t* __restrict__ idx, int64_t M, int32_t n_adapters, int64_t tiles512, AdapterLists l,
            uint32_t* err) {
    extern __shared__ int32_t table[];            // [n_adapters] first token of the tile, up to kTableAdapters
    grid_dependency_wait();
    allow_dependents();
    __shared__ __align__(16) int32_t ids[512];
    __shared__ int32_t slot[512];
    __shared__ uint32_t ballots[kGradBatch][16];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    if (blockIdx.x >= tiles512) {
        const int32_t a = (int32_t)(blockIdx.x - tiles512);
        uint4* out = l.e_grad + (int64_t)a * l.tiles64;
        int32_t found = 0;
        for (int64_t m0 = 0; m0 < M; m0 += 512 * kGradBatch) {
            bool mine[kGradBatch];
#pragma unroll
            for (int k = 0; k < kGradBatch; ++k) mine[k] = m0 + 512 * k + t < M && idx[m0 + 512 * k + t] == a;
#pragma unroll
            for (int k = 0; k < kGradBatch; ++k) {
                const uint32_t b = __ballot_sync(0xffffffffu, mine[k]);
                if (lane == 0) ballots[k][warp] = b;
            }
            __syncthreads();
            if (warp == 0) {                                  // lane i: the token tile i of the batch
                const uint32_t* w = &ballots[0][0] + 2 * lane;
                const bool any = (w[0] | w[1]) != 0;
                const uint32_t tiles = __ballot_sync(0xffffffffu, any);
                if (any) {
                    const int64_t left = M - (m0 + 64 * lane);    // rows of this token tile
                    const uint32_t lo = left >= 32 ? 0xffffffffu : (1u << left) - 1u;
                    const uint32_t hi = left >= 64 ? 0xffffffffu : left > 32 ? (1u << (left - 32)) - 1u : 0u;
                    out[found + __popc(tiles & ((1u << lane) - 1u))] =
                        make_uint4((uint32_t)(m0 / 64 + lane), w[0], w[1], (w[0] == lo && w[1] == hi) ? 1u : 0u);
                }
                found += __popc(tiles);
            }
            __syncthreads();
        }
        if (t == 0) l.n_grad[a] = (uint32_t)found;
        return;
    }
    const bool tabled = n_adapters <= kTableAdapters;
    const int64_t m = (int64_t)blockIdx.x * 512 + t;
    int32_t a = m < M ? idx[m] : -1;
    if (a >= n_adapters) {
        atomicOr(err, ERR_FLAG_BOUNDS);
        a = -1;
    }
    if (a < 0) a = -1;
    if (m < M) l.tok[m] = a;
    if (tabled)
        for (int i = t; i < n_adapters; i += 512) table[i] = 512;
    else
        ids[t] = a;
    __syncthreads();
    const uint32_t same = __match_any_sync(0xffffffffu, a);
    const bool leads = a >= 0 && lane == __ffs((int)same) - 1;   // the warp's first token with the adapter
    int f512 = t;
    if (tabled) {
        if (leads) atomicMin(table + a, t);
        __syncthreads();
        if (a >= 0) f512 = table[a];
    } else {
        for (int j = t & ~3; j >= 0; j -= 4) {
            const int4 v = *reinterpret_cast<const int4*>(ids + j);
            const int f = v.x == a ? j : v.y == a ? j + 1 : v.z == a ? j + 2 : v.w == a ? j + 3 : 512;
            f512 = min(f512, f);
        }
    }
    const bool first = a >= 0 && f512 == t;
    const uint32_t b = __ballot_sync(0xffffffffu, first);
    if (lane == 0) ballots[0][warp] = b;
    __syncthreads();
    int before = __popc(b & ((1u << lane) - 1u)), total = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        const int c = __popc(ballots[0][w]);
        if (w < warp) before += c;
        total += c;
    }
    uint32_t* e512 = l.e512 + (int64_t)blockIdx.x * l.cap512 * kAdEntry;
    if (t == 0) l.n512[blockIdx.x] = (uint32_t)total;
    if (first) {
        slot[t] = before;
        uint4* e = reinterpret_cast<uint4*>(e512 + (int64_t)before * kAdEntry);
#pragma unroll
        for (int q = 0; q < 4; ++q) e[q] = make_uint4(0, 0, 0, 0);
        e[4] = make_uint4((uint32_t)a, 0, 0, 0);
    }
    __syncthreads();
    if (leads) e512[slot[f512] * kAdEntry + warp] = same;
}

// ---------------------------------------------------------------------------- U and dU

// partial[split][m][0 .. Rn) = sum over the split's 64-wide reduction steps of S[m] . V_a[j], S = X
// with V = A_all (reduction over K), or S = dY with V = B_all (reduction over N, V MN-major).
// CTA (token tile of 128, split): each reduction step loads the S tile once and one tile of V for each
// adapter of the tile; the adapter's MMA writes its own rows of the one accumulator.  Rows without an
// adapter are written as zeros.  Two rings, so that one S tile serves many V tiles.
// Roles (192 threads): warp 0 TMA, warp 1 TMEM owner + MMA issuer, warps 2-5 epilogue.
constexpr int kPartThreads = 192;

struct PartParams {
    int64_t M;
    int32_t Rn;               // ranks rounded up to 16: columns of the accumulator
    int32_t ksteps_total, ksteps_per_split;
    uint32_t tmem_cols, s_stages, v_stages, v_tile;
    int32_t f16;
    const uint32_t* count;
    const uint32_t* entry;
    int32_t cap;
    const int32_t* tok;
    float* partial;
    uint32_t* err;
};

struct PartLayout {
    uint32_t off_v, off_mask, off_adapter, off_bars, off_slot, off_abort, off_count, alloc;
};
__host__ __device__ inline PartLayout part_layout(uint32_t s_stages, uint32_t v_stages, uint32_t v_tile) {
    PartLayout l;
    l.off_v = s_stages * kStage16K;
    l.off_mask = l.off_v + v_stages * v_tile;
    l.off_adapter = l.off_mask + 128 * 16;
    l.off_bars = l.off_adapter + 128 * 4;
    l.off_slot = l.off_bars + (2 * s_stages + 2 * v_stages + 1) * 8;
    l.off_abort = l.off_slot + 4;
    l.off_count = l.off_abort + 4;
    l.alloc = l.off_count + 4 + 1024;
    return l;
}

template <bool V_MN>
__global__ void __launch_bounds__(kPartThreads, 2)
tc_part_gemm(const __grid_constant__ CUtensorMap tmS, const __grid_constant__ CUtensorMap tmV, PartParams p) {
    grid_dependency_wait();
    allow_dependents();
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - ptx::smem_addr(smem_raw));
    const PartLayout lay = part_layout(p.s_stages, p.v_stages, p.v_tile);
    const int SS = (int)p.s_stages, VS = (int)p.v_stages;
    const uint32_t sS = base, sV = base + lay.off_v;
    const uint32_t bar_sfull = base + lay.off_bars, bar_sempty = bar_sfull + 8 * SS;
    const uint32_t bar_vfull = bar_sempty + 8 * SS, bar_vempty = bar_vfull + 8 * VS;
    const uint32_t bar_acc = bar_vempty + 8 * VS;
    uint4* mask = reinterpret_cast<uint4*>(gbase + lay.off_mask);
    int32_t* adapter = reinterpret_cast<int32_t*>(gbase + lay.off_adapter);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + lay.off_slot);
    volatile int* abort = reinterpret_cast<volatile int*>(gbase + lay.off_abort);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row0 = (int64_t)blockIdx.x * kPartTile;
    const int k_begin = blockIdx.y * p.ksteps_per_split;
    const int k_end = min(p.ksteps_total, k_begin + p.ksteps_per_split);
    volatile int32_t* n_ads = reinterpret_cast<volatile int32_t*>(gbase + lay.off_count);
    if (warp == 2) {                                          // the entries of the 512-token tile that reach this 128
        const int64_t t512 = row0 / kAdTile;
        const int listed = (int)p.count[t512];
        const uint32_t* e = p.entry + t512 * p.cap * kAdEntry;
        int found = 0;
        for (int i0 = 0; i0 < listed; i0 += 32) {
            uint4 v = make_uint4(0, 0, 0, 0);
            int32_t a = 0;
            if (i0 + lane < listed) {
                const uint32_t* at = e + (int64_t)(i0 + lane) * kAdEntry;
                v = *reinterpret_cast<const uint4*>(at + (row0 % kAdTile) / 32);
                a = (int32_t)at[16];
            }
            const bool here = (v.x | v.y | v.z | v.w) != 0;
            const uint32_t all = __ballot_sync(0xffffffffu, here);
            if (here) {
                const int at = found + __popc(all & ((1u << lane) - 1u));
                mask[at] = make_uint4(~v.x, ~v.y, ~v.z, ~v.w);
                adapter[at] = a;
            }
            found += __popc(all);
        }
        if (lane == 0) *n_ads = found;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < SS; ++s) {
            ptx::mbar_init(bar_sfull + 8 * s, 1);
            ptx::mbar_init(bar_sempty + 8 * s, 1);
        }
        for (int s = 0; s < VS; ++s) {
            ptx::mbar_init(bar_vfull + 8 * s, 1);
            ptx::mbar_init(bar_vempty + 8 * s, 1);
        }
        ptx::mbar_init(bar_acc, 1);
        *abort = 0;
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_smem();
        ptx::tma_prefetch_map(&tmS);
        ptx::tma_prefetch_map(&tmV);
    }
    if (warp == 1) {
        ptx::tmem_alloc(base + lay.off_slot, p.tmem_cols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int n_ad = *n_ads, nk = n_ad > 0 ? k_end - k_begin : 0;

    if (warp == 0) {
        int s = 0, v = 0, s_issued = 0, v_issued = 0;
        uint32_t s_ph = 0, v_ph = 0;
        bool ok = true;
        for (int i = 0; i < nk && ok; ++i) {
            const int ks = k_begin + i;
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_sempty + 8 * s, s_ph ^ 1u, abort, p.err));
            if (!ok) break;
            if (ptx::elect_one_sync()) {
                ptx::mbar_arrive_expect_tx(bar_sfull + 8 * s, kStage16K);
                ptx::tma_load_2d(sS + s * kStage16K, &tmS, ks * 64, (int32_t)row0, bar_sfull + 8 * s);
            }
            __syncwarp();
            ++s_issued;
            if (++s == SS) { s = 0; s_ph ^= 1u; }
            for (int e = 0; e < n_ad; ++e) {
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_vempty + 8 * v, v_ph ^ 1u, abort, p.err));
                if (!ok) break;
                if (ptx::elect_one_sync()) {
                    const uint32_t fb = bar_vfull + 8 * v, dst = sV + v * p.v_tile;
                    ptx::mbar_arrive_expect_tx(fb, p.v_tile);
                    if (!V_MN) {
                        ptx::tma_load_3d(dst, &tmV, ks * 64, 0, adapter[e], fb);
                    } else {
                        for (uint32_t c = 0; c * 8192u < p.v_tile; ++c)
                            ptx::tma_load_3d(dst + c * 8192u, &tmV, (int32_t)c * 64, ks * 64, adapter[e], fb);
                    }
                }
                __syncwarp();
                ++v_issued;
                if (++v == VS) { v = 0; v_ph ^= 1u; }
            }
        }
        if (*abort) {   // drain this CTA's copies in flight before it exits
            for (int c = max(0, s_issued - SS); c < s_issued; ++c)
                ptx::mbar_wait_drain(bar_sfull + 8 * (c % SS), (uint32_t)(c / SS) & 1u);
            for (int c = max(0, v_issued - VS); c < v_issued; ++c)
                ptx::mbar_wait_drain(bar_vfull + 8 * (c % VS), (uint32_t)(c / VS) & 1u);
        }
    } else if (warp == 1) {
        const uint32_t idesc = ptx::idesc_set_f16(ptx::idesc_bf16_f32_ab(128, p.Rn, 0, V_MN ? 1 : 0), p.f16 != 0);
        int s = 0, v = 0;
        uint32_t s_ph = 0, v_ph = 0;
        bool ok = true;
        for (int i = 0; i < nk && ok; ++i) {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_sfull + 8 * s, s_ph, abort, p.err));
            for (int e = 0; e < n_ad && ok; ++e) {
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_vfull + 8 * v, v_ph, abort, p.err));
                if (!ok) break;
                ptx::tc_fence_after();
                const uint4 mk = mask[e];
                const uint32_t off[4] = {mk.x, mk.y, mk.z, mk.w};
                if (ptx::elect_one_sync()) {
                    const uint32_t a_base = sS + s * kStage16K, b_base = sV + v * p.v_tile;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        ptx::mma_bf16_ss_lanes(tmem, ptx::smem_desc_sw128(a_base + kk * 32, 16, 1024),
                                               V_MN ? ptx::smem_desc_sw128(b_base + kk * 2048, 8192, 1024)
                                                    : ptx::smem_desc_sw128(b_base + kk * 32, 16, 1024),
                                               idesc, (i | kk) != 0 ? 1u : 0u, off);
                    ptx::mma_commit(bar_vempty + 8 * v);
                    if (e == n_ad - 1) ptx::mma_commit(bar_sempty + 8 * s);
                }
                __syncwarp();
                if (++v == VS) { v = 0; v_ph ^= 1u; }
            }
            if (++s == SS) { s = 0; s_ph ^= 1u; }
        }
        if (ptx::elect_one_sync()) {
            ptx::mma_commit(bar_acc);
            if (*abort) ptx::mbar_wait_drain(bar_acc, 0);   // issued MMAs finish before TMEM is freed
        }
        __syncwarp();
    } else {
        const bool acc_ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_acc, 0, abort, p.err));
        ptx::tc_fence_after();
        if (acc_ok) {
            const uint32_t quad = (uint32_t)(warp & 3);
            const int64_t row = row0 + quad * 32 + lane;
            const bool have = row < p.M && nk > 0 && p.tok[row] >= 0;
            float* dst = p.partial + ((int64_t)blockIdx.y * p.M + row) * p.Rn;
#pragma unroll 1
            for (int c = 0; c < p.Rn / 16; ++c) {
                uint32_t v[16];
                ptx::tmem_ld_32x32b_x16(tmem + ((quad * 32u) << 16) + c * 16, v);
                ptx::tmem_ld_wait();
                if (row < p.M) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = have ? v[i] : 0u;
                    store_sector(dst + c * 16, v);
                    store_sector(dst + c * 16 + 8, v + 8);
                }
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, p.tmem_cols);
    }
}

// V[m, j] = the sum of the splits' partials, in split order (out, fp32 [M, r]; may be null), and s_a V[m, j]
// as sums of 16-bit numbers of the compute type t, which the tensor cores need (zeros for j >= r and for
// tokens without an adapter):
//   V2 [M, 2R] (may be null): hi = t(v) and lo = t(v - hi), for the products that are rounded to 16 bits
//   after them; together within 2^-17 of v in bf16.
//   V3 [M, 3 Rg] (may be null): three parts, for the fp32 gradients; together within 2^-24 of v.  In fp16
//   the second and third are kept 2^11 and 2^22 times too large, which their own accumulators undo:
//   the residuals of a small gradient would otherwise fall below the type's range.  Ranks come in
//   blocks of RB, each [part][RB].
// With splits = 0 the values are V itself (a saved U, [M, r]).  Blocks of y = 1 do the same for a second
// source.
struct FinishSource {
    const float* from;
    int splits;
    float* out;
    uint16_t* V2;
    uint16_t* V3;
};
constexpr float kPartScale = 2048.f;              // 2^11, fp16

__global__ void __launch_bounds__(256)
finish_part(FinishSource s0, FinishSource s1, int64_t M, int r, int Rn, int R, int RB, int Rg,
            const int32_t* __restrict__ tok, const float* __restrict__ scales, bool f16) {
    grid_dependency_wait();
    allow_dependents();
    const FinishSource& f = blockIdx.y == 0 ? s0 : s1;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= M * Rg) return;
    const int64_t m = i / Rg;
    const int j = (int)(i - m * Rg);
    const int32_t a = tok[m];
    float v = 0.f, sv = 0.f;
    if (j < r && a >= 0) {
        const float scale = __ldg(scales + a);
        if (f.splits == 0) {
            v = f.from[m * r + j];
        } else {
            const int64_t stride = M * Rn;
            const float* q = f.from + m * Rn + j;
            int s = 0;
            for (; s + 8 <= f.splits; s += 8) {
                float w[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) w[u] = q[(s + u) * stride];
#pragma unroll
                for (int u = 0; u < 8; ++u) v = __fadd_rn(v, w[u]);
            }
            for (; s < f.splits; ++s) v = __fadd_rn(v, q[s * stride]);
        }
        sv = __fmul_rn(scale, v);
    }
    if (f.out && j < r) f.out[m * r + j] = v;
    const uint32_t hi = to16_rn(sv, f16);
    const float rest = __fsub_rn(sv, from16(hi, f16));
    if (f.V2 && j < R) {
        f.V2[m * 2 * R + j] = (uint16_t)hi;
        f.V2[m * 2 * R + R + j] = (uint16_t)to16_rn(rest, f16);
    }
    if (f.V3) {
        const float up = f16 ? kPartScale : 1.f;              // powers of two: exact
        const uint32_t mid = to16_rn(__fmul_rn(rest, up), f16);
        const float last = __fsub_rn(__fmul_rn(rest, up), from16(mid, f16));
        uint16_t* at = f.V3 + m * 3 * Rg + (j / RB) * 3 * RB + j % RB;
        at[0] = (uint16_t)hi;
        at[RB] = (uint16_t)mid;
        at[2 * RB] = (uint16_t)to16_rn(__fmul_rn(last, up), f16);
    }
}

// ---------------------------------------------------------------------------- dA and dB

// dA_a^T[k, j] = sum over the adapter's tokens of X[m, k] dU[m, j], and dB_a[n, j] likewise of dY and
// s_a U, in one launch: CTA (x, a, z) computes 128 rows k (or n) and rank block z of adapter a over the
// adapter's token tiles.  Operand A is the [64 tokens x 128] tile of X or dY (MN-major), operand B the
// three parts of dU or s U side by side, each with an accumulator of its own (one MMA of N = 3 RB, or one
// of N = RB for each part when that exceeds 256); the epilogue adds the parts in fp32.
// Roles (192 threads): warp 0 TMA, warp 1 TMEM owner + MMA issuer, warps 2-5 zero the rows of other
// tokens in tiles that the adapter shares, then run the epilogue.
// Every 8 token tiles the accumulators are added to the output and begun anew: the tensor cores' fp32
// sums lose about 2^-26 of themselves at each 16-wide step, one way, which a long batch would notice.  dB of
// 2000 tokens of two adapters is off by 6.0e-7 (in tiles of 16: 1.1e-6; a plain fp32 sum: 3.9e-7), for 1% of a
// training step of 2048 tokens, W[8192, 8192] (500 to 506 us); 4 tiles give 3.3e-7 for another 3%.
constexpr int kGradThreads = 192;
constexpr int kGradFlush = 8;

struct GradParams {
    int64_t M, K, N;
    int32_t r, RB;            // ranks, and ranks of a block (z)
    int32_t tiles_k;          // CTAs x < tiles_k compute dA, the others dB
    uint32_t stages, v_bytes, tmem_cols;
    int32_t f16;
    const uint32_t* n_grad;
    const uint4* e_grad;
    int32_t tiles64;
    float* dA;                // [n, r, K]
    float* dB;                // [n, N, r]
    uint32_t* err;
};

struct GradLayout {
    uint32_t off_v, off_bars, off_slot, off_abort, alloc;
};
__host__ __device__ inline GradLayout grad_layout(uint32_t stages, uint32_t v_bytes) {
    GradLayout l;
    l.off_v = stages * kStage16K;
    l.off_bars = l.off_v + stages * v_bytes;
    l.off_slot = l.off_bars + (3 * stages + 2) * 8;
    l.off_abort = l.off_slot + 4;
    l.alloc = l.off_abort + 4 + 1024;
    return l;
}

__global__ void __launch_bounds__(kGradThreads, 2)
tc_adapter_grads(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmdY,
                 const __grid_constant__ CUtensorMap tmdU3, const __grid_constant__ CUtensorMap tmU3, GradParams p) {
    grid_dependency_wait();
    allow_dependents();
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - ptx::smem_addr(smem_raw));
    const GradLayout lay = grad_layout(p.stages, p.v_bytes);
    const int S = (int)p.stages;
    const uint32_t sS = base, sV = base + lay.off_v;
    const uint32_t bar_full = base + lay.off_bars, bar_ready = bar_full + 8 * S, bar_empty = bar_ready + 8 * S;
    const uint32_t bar_acc = bar_empty + 8 * S, bar_flushed = bar_acc + 8;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + lay.off_slot);
    volatile int* abort = reinterpret_cast<volatile int*>(gbase + lay.off_abort);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool is_a = (int)blockIdx.x < p.tiles_k;
    const int64_t row0 = (int64_t)(is_a ? blockIdx.x : blockIdx.x - p.tiles_k) * 128;
    const int32_t ad = (int32_t)blockIdx.y;
    const int nt = (int)p.n_grad[ad];
    const uint4* list = p.e_grad + (int64_t)ad * p.tiles64;
    const int chunks = (int)(p.v_bytes / 8192);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_ready + 8 * s, 4);
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        ptx::mbar_init(bar_acc, 1);
        ptx::mbar_init(bar_flushed, 4);
        *abort = 0;
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 1) {
        ptx::tmem_alloc(base + lay.off_slot, p.tmem_cols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        int s = 0, issued = 0;
        uint32_t ph = 0;
        int32_t tile = nt > 0 ? (int32_t)__ldg(&list[0].x) : 0;
        for (int i = 0; i < nt; ++i) {
            const int32_t next = i + 1 < nt ? (int32_t)__ldg(&list[i + 1].x) : 0;
            if (!__all_sync(0xffffffffu, ptx::mbar_wait(bar_empty + 8 * s, ph ^ 1u, abort, p.err))) break;
            issued = i + 1;
            if (ptx::elect_one_sync()) {
                const uint32_t fb = bar_full + 8 * s, s_dst = sS + s * kStage16K, v_dst = sV + s * p.v_bytes;
                const CUtensorMap* ms = is_a ? &tmX : &tmdY;
                const CUtensorMap* mv = is_a ? &tmdU3 : &tmU3;
                ptx::mbar_arrive_expect_tx(fb, kStage16K + p.v_bytes);
                ptx::tma_load_2d(s_dst, ms, (int32_t)row0, tile * kGradTile, fb);
                ptx::tma_load_2d(s_dst + 8192, ms, (int32_t)row0 + 64, tile * kGradTile, fb);
                for (int c = 0; c < chunks; ++c)
                    ptx::tma_load_2d(v_dst + c * 8192, mv, (int32_t)blockIdx.z * 3 * p.RB + c * 64, tile * kGradTile, fb);
            }
            __syncwarp();
            tile = next;
            if (++s == S) { s = 0; ph ^= 1u; }
        }
        if (*abort) {   // drain this CTA's copies in flight before it exits
            for (int i = max(0, issued - S); i < issued; ++i)
                ptx::mbar_wait_drain(bar_full + 8 * (i % S), (uint32_t)(i / S) & 1u);
        }
    } else if (warp == 1) {
        const bool side = 3 * p.RB <= 256;                    // all parts in one MMA
        const uint32_t idesc =
            ptx::idesc_set_f16(ptx::idesc_bf16_f32_ab(128, side ? 3 * p.RB : p.RB, 1, 1), p.f16 != 0);
        int s = 0;
        uint32_t ph = 0, acc_ph = 0;                          // phase of bar_acc that the next commit completes
        bool ok = true;
        for (int i = 0; i < nt && ok; ++i) {
            const bool fresh = i % kGradFlush == 0;
            bool w = true;
            if (fresh && i > 0) w = ptx::mbar_wait(bar_flushed, (uint32_t)(i / kGradFlush - 1) & 1u, abort, p.err);
            ok = __all_sync(0xffffffffu, w && ptx::mbar_wait(bar_ready + 8 * s, ph, abort, p.err));
            if (!ok) break;
            ptx::tc_fence_after();
            if (ptx::elect_one_sync()) {
                const uint32_t a_base = sS + s * kStage16K, b_base = sV + s * p.v_bytes;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint64_t ad_desc = ptx::smem_desc_sw128(a_base + kk * 2048, 8192, 1024);
                    for (int part = 0; part < (side ? 1 : 3); ++part)
                        ptx::mma_bf16_ss(tmem + (uint32_t)(part * p.RB), ad_desc,
                                         ptx::smem_desc_sw128(b_base + part * (p.RB / 64) * 8192 + kk * 2048, 8192, 1024),
                                         idesc, (fresh && kk == 0) ? 0u : 1u);
                }
                ptx::mma_commit(bar_empty + 8 * s);
                if ((i + 1) % kGradFlush == 0 && i + 1 < nt) ptx::mma_commit(bar_acc);
            }
            __syncwarp();
            if ((i + 1) % kGradFlush == 0 && i + 1 < nt) acc_ph ^= 1u;
            if (++s == S) { s = 0; ph ^= 1u; }
        }
        if (ptx::elect_one_sync()) {
            ptx::mma_commit(bar_acc);
            if (*abort) ptx::mbar_wait_drain(bar_acc, acc_ph);   // issued MMAs finish before TMEM is freed
        }
        __syncwarp();
    } else {
        const int t = threadIdx.x - 64, row = t & 63, half = t >> 6;
        const uint32_t quad = (uint32_t)(warp & 3);
        const int64_t orow = row0 + quad * 32 + lane;
        const bool in = orow < (is_a ? p.K : p.N);
        const int j0 = (int)blockIdx.z * p.RB, nj = min(p.r - j0, p.RB);
        float* const dst = is_a ? p.dA + ((int64_t)ad * p.r + j0) * p.K + orow : p.dB + ((int64_t)ad * p.N + orow) * p.r + j0;
        const int64_t pitch = is_a ? p.K : 1;                 // between a thread's ranks
        const bool vec = !is_a && p.r % 4 == 0;
        const bool sectors = !is_a && p.r % 8 == 0 && (reinterpret_cast<uintptr_t>(p.dB) & 31u) == 0;
        const float down = p.f16 ? 1.f / kPartScale : 1.f;
        // the accumulators of piece f of the token tiles, stored (f = 0) or added to what the thread stored
        auto flush = [&](int f) -> bool {
            const bool acc_ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_acc, (uint32_t)f & 1u, abort, p.err));
            if (!acc_ok) return false;
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c * 16 < nj; ++c) {
                float v[16];
                if (nt > 0) {
                    uint32_t part[3][16];
#pragma unroll
                    for (int w = 0; w < 3; ++w)
                        ptx::tmem_ld_32x32b_x16(tmem + ((quad * 32u) << 16) + (uint32_t)(w * p.RB + c * 16), part[w]);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        v[q] = __fmaf_rn(__fmaf_rn(__uint_as_float(part[2][q]), down, __uint_as_float(part[1][q])), down,
                                         __uint_as_float(part[0][q]));
                } else {                                      // no token has this adapter
#pragma unroll
                    for (int q = 0; q < 16; ++q) v[q] = 0.f;
                }
                if (!in) continue;
                float* at = dst + (int64_t)c * 16 * pitch;
                if (f > 0)
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        if (c * 16 + q < nj) v[q] = __fadd_rn(at[q * pitch], v[q]);
                if (sectors) {
                    uint32_t w[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q) w[q] = __float_as_uint(v[q]);
                    store_sector(at, w);
                    if (c * 16 + 8 < nj) store_sector(at + 8, w + 8);
                } else if (vec) {
#pragma unroll
                    for (int q = 0; q < 16; q += 4)
                        if (c * 16 + q < nj) *reinterpret_cast<float4*>(at + q) = make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
                } else {
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        if (c * 16 + q < nj) at[q * pitch] = v[q];
                }
            }
            return true;
        };
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        uint4 e = nt > 0 ? __ldg(list) : make_uint4(0, 0, 0, 0);
        for (int i = 0; i < nt && ok; ++i) {
            const uint4 next = i + 1 < nt ? __ldg(list + i + 1) : make_uint4(0, 0, 0, 0);
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_full + 8 * s, ph, abort, p.err));
            if (!ok) break;
            if (e.w == 0u) {
                const bool mine = ((row < 32 ? e.y : e.z) >> (row & 31)) & 1u;
                if (!mine) {   // a token is one 128-byte row of every image
                    const uint32_t x = sS + s * kStage16K + half * 8192u + row * 128u;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(x + 16 * c), "r"(0) : "memory");
                    for (int q = half; q < chunks; q += 2) {
                        const uint32_t v = sV + s * p.v_bytes + q * 8192u + row * 128u;
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(v + 16 * c), "r"(0) : "memory");
                    }
                }
                ptx::fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_ready + 8 * s);
            e = next;
            if (++s == S) { s = 0; ph ^= 1u; }
            if ((i + 1) % kGradFlush == 0 && i + 1 < nt) {
                ok = flush(i / kGradFlush);
                if (!ok) break;
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar_flushed);
            }
        }
        if (ok) (void)flush(nt > 0 ? (nt - 1) / kGradFlush : 0);
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, p.tmem_cols);
    }
}

// out[i, 0 .. cols_out) = in[i, 0 .. cols) and zeros: 16-bit rows brought to a multiple of 16 bytes,
// which TMA needs of its row strides (B_all with r % 8 != 0, dY with N % 8 != 0).
__global__ void __launch_bounds__(256)
pad_rows(const uint16_t* __restrict__ in, int64_t rows, int64_t cols, int64_t cols_out, uint4* __restrict__ out) {
    grid_dependency_wait();
    allow_dependents();
    const int64_t chunks = cols_out / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= rows * chunks) return;
    const int64_t row = i / chunks, c = (i - row * chunks) * 8;
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int64_t j = c + 2 * q;
        const uint32_t lo = j < cols ? in[row * cols + j] : 0u, hi = j + 1 < cols ? in[row * cols + j + 1] : 0u;
        w[q] = lo | (hi << 16);
    }
    out[i] = make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------------------- host

inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Half width of the hi/lo operands: 32 (both halves share one 64-wide step) or a multiple of 64.
inline int32_t half_width(int32_t r) { return r <= 32 ? 32 : (int32_t)round_up(r, 64); }

// Ranks of a block of the gradients' three-part operands: 32, 64 or 128, and all blocks' ranks.
inline int32_t grad_block(int32_t r) { return r <= 32 ? 32 : r <= 64 ? 64 : 128; }
inline int32_t grad_ranks(int32_t r) { return (int32_t)round_up(r, grad_block(r)); }

// Workspace, every piece 256-byte aligned:
//   the lists; V2, 16-bit [M, 2R] (hi | lo of s U in the forward, of dU in the backward); U3 and dU3,
//   16-bit [M, 3 Rg] (three parts of s U and of dU); partial, fp32 (splits of U or dU, or the small-M
//   forward's partial tiles); split, fp32 partial outputs of a split reduction; B8, B_all with its rows
//   padded to 16 bytes (r % 8 != 0); dY8 likewise (N % 8 != 0).
struct AdaptersWs {
    size_t tok, n512, e512, n_grad, e_grad, v2, u3, du3, part, split, b8, dy8, total;
    size_t split_bytes;
    int32_t cap512, tiles64;
    int64_t tiles512;
};

// Splits of the reduction of U or dU: two CTAs for each of 148 SMs (a count fixed here, so that the
// workspace does not depend on the current device) while each has at least two steps of 64, and no more
// than 16 steps each: the tensor cores' fp32 sums lose about 2^-27 of themselves at every 16-wide step,
// one way.  Rounded so that no split is empty.
int part_splits(int64_t M, int64_t red, int32_t r) {
    const int64_t tiles = (M + kPartTile - 1) / kPartTile, steps = (red + 63) / 64;
    const int64_t most = r <= 128 ? 2 * 148 : 148;            // CTAs that run together
    const int64_t want = std::max<int64_t>((steps + 15) / 16, std::min(most / tiles, steps / 2));
    const int64_t per = (steps + want - 1) / want;
    return (int)((steps + per - 1) / per);
}

AdaptersWs adapters_ws(int64_t M, int64_t N, int64_t K, int32_t r, int64_t n) {
    AdaptersWs w;
    const int64_t R = half_width(r), Rn = round_up(r, 16);
    w.tiles512 = (M + kAdTile - 1) / kAdTile;
    w.cap512 = (int32_t)std::min<int64_t>({(int64_t)kAdTile, n, M});
    w.tiles64 = (int32_t)((M + 63) / 64);
    size_t o = 0;
    auto piece = [&o](size_t bytes) { const size_t at = o; o += align_up(bytes, 256); return at; };
    w.tok = piece(M * 4);
    w.n512 = piece(w.tiles512 * 4);
    w.e512 = piece((size_t)w.tiles512 * w.cap512 * kAdEntry * 4);
    w.n_grad = piece(n * 4);
    w.e_grad = piece((size_t)n * w.tiles64 * 16);
    w.v2 = piece((size_t)M * 2 * R * 2);
    w.u3 = piece((size_t)M * 3 * grad_ranks(r) * 2);
    w.du3 = piece((size_t)M * 3 * grad_ranks(r) * 2);
    size_t part = (size_t)std::max(part_splits(M, K, r), part_splits(M, N, r)) * M * Rn * 4;
    if (M <= kRowsMaxM) part = std::max(part, rows_workspace_bytes(M, N, K, r, n));
    w.part = piece(part);
    w.split_bytes = std::max(M > kRowsMaxM ? adapters_split_bytes(M, N, K, false) : 0, adapters_split_bytes(M, N, K, true));
    w.split = piece(w.split_bytes);
    w.b8 = piece(r % 8 ? (size_t)n * N * round_up(r, 8) * 2 : 0);
    w.dy8 = piece(N % 8 ? (size_t)M * round_up(N, 8) * 2 : 0);
    w.total = o + 256;                                        // the caller's pointer is brought to 256 bytes
    return w;
}

AdapterLists lists_at(char* ws, const AdaptersWs& w) {
    AdapterLists l;
    l.tok = reinterpret_cast<int32_t*>(ws + w.tok);
    l.n512 = reinterpret_cast<uint32_t*>(ws + w.n512);
    l.e512 = reinterpret_cast<uint32_t*>(ws + w.e512);
    l.n_grad = reinterpret_cast<uint32_t*>(ws + w.n_grad);
    l.e_grad = reinterpret_cast<uint4*>(ws + w.e_grad);
    l.cap512 = w.cap512; l.tiles64 = w.tiles64;
    return l;
}

qlora_status launch_lists(const int32_t* idx, int64_t M, int32_t n, const AdaptersWs& w, const AdapterLists& l,
                          bool grads, cudaStream_t s) {
    uint32_t* err = device_error_word();
    if (!err) return QLORA_ERR_CUDA;
    const size_t table = n <= kTableAdapters ? (size_t)n * 4 : 0;
    (void)launch_dependent(build_lists, dim3((unsigned)(w.tiles512 + (grads ? n : 0))), dim3(512), table, s, idx, M, n,
                           w.tiles512, l, err);
    QLORA_CHECK_LAUNCH();
    return QLORA_OK;
}

qlora_status launch_pad_rows(const void* in, int64_t rows, int64_t cols, void* out, cudaStream_t s) {
    const int64_t cols_out = round_up(cols, 8), blocks = (rows * (cols_out / 8) + 255) / 256;
    if (blocks > INT32_MAX) return QLORA_ERR_SHAPE;
    (void)launch_dependent(pad_rows, dim3((unsigned)blocks), dim3(256), 0, s, static_cast<const uint16_t*>(in), rows,
                           cols, cols_out, static_cast<uint4*>(out));
    QLORA_CHECK_LAUNCH();
    return QLORA_OK;
}

template <bool V_MN>
qlora_status launch_part(const CUtensorMap& tmS, const CUtensorMap& tmV, PartParams& p, int splits, cudaStream_t s) {
    static std::atomic<uint64_t> configured{0};
    auto kern = tc_part_gemm<V_MN>;
    if (!allow_smem(configured, (const void*)kern, (int)kMaxSmem)) return QLORA_ERR_CUDA;
    // two CTAs per SM up to 128 ranks: three S stages and the rest of 108 KiB for V tiles, of which a tile of
    // many adapters takes many per S tile
    p.s_stages = 3;
    p.v_stages = std::min(16u, std::max(3u, (108u * 1024 - p.s_stages * kStage16K) / p.v_tile));
    const PartLayout lay = part_layout(p.s_stages, p.v_stages, p.v_tile);
    if (lay.alloc > kMaxSmem) return QLORA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)((p.M + kPartTile - 1) / kPartTile), (unsigned)splits);
    (void)launch_dependent(kern, grid, dim3(kPartThreads), lay.alloc, s, tmS, tmV, p);
    QLORA_CHECK_LAUNCH();
    return QLORA_OK;
}

// partial = S V_a^T over the adapters: S [M, red] 16-bit with rows of ld elements; V = A_all
// [n, r, red] (v_mn false) or B_all [n, red, ldv] with r of its ldv columns (v_mn true).
// Returns the split count in *splits_out.
qlora_status part_gemm(const void* S, int64_t M, int64_t red, int64_t ld, const void* V, bool v_mn, int64_t ldv,
                       int32_t r, int32_t n, const AdapterLists& l, float* partial, bool f16, int* splits_out,
                       cudaStream_t s) {
    PartParams p{};
    p.M = M;
    p.Rn = (int32_t)round_up(r, 16);
    p.ksteps_total = (int32_t)((red + 63) / 64);
    const int splits = part_splits(M, red, r);
    p.ksteps_per_split = (p.ksteps_total + splits - 1) / splits;
    p.tmem_cols = p.Rn <= 32 ? 32u : p.Rn <= 64 ? 64u : p.Rn <= 128 ? 128u : 256u;
    p.v_tile = v_mn ? (uint32_t)round_up(p.Rn, 64) * 128u : (uint32_t)p.Rn * 128u;
    p.v_tile = (uint32_t)round_up(p.v_tile, 1024);            // swizzle atoms stay aligned
    p.f16 = f16;
    p.count = l.n512; p.entry = l.e512; p.cap = l.cap512; p.tok = l.tok;
    p.partial = partial;
    p.err = device_error_word();
    if (!p.err) return QLORA_ERR_CUDA;
    *splits_out = splits;
    CUtensorMap tmS, tmV;
    if (!make_tmap_2d(&tmS, true, S, red, M, ld * 2, 64, 128, true)) return QLORA_ERR_CUDA;
    if (v_mn) {
        if (!make_tmap_3d(&tmV, V, ldv, red, n, 64, 64)) return QLORA_ERR_CUDA;
        return launch_part<true>(tmS, tmV, p, splits, s);
    }
    if (!make_tmap_3d(&tmV, V, red, r, n, 64, (uint32_t)p.Rn)) return QLORA_ERR_CUDA;
    return launch_part<false>(tmS, tmV, p, splits, s);
}

// One source, or two (s1.V3 set).
qlora_status launch_finish(const FinishSource& s0, const FinishSource& s1, int64_t M, int32_t r, const AdapterLists& l,
                           const float* scales, bool f16, cudaStream_t s) {
    const int64_t blocks = (M * grad_ranks(r) + 255) / 256;
    if (blocks > INT32_MAX) return QLORA_ERR_SHAPE;
    (void)launch_dependent(finish_part, dim3((unsigned)blocks, s1.V3 ? 2u : 1u), dim3(256), 0, s, s0, s1, M, (int)r,
                           (int)round_up(r, 16), (int)half_width(r), (int)grad_block(r), (int)grad_ranks(r),
                           (const int32_t*)l.tok, scales, f16);
    QLORA_CHECK_LAUNCH();
    return QLORA_OK;
}

qlora_status launch_grads(const void* X, const void* dY, int64_t ldy, int64_t M, int64_t N, int64_t K, int32_t r,
                          int32_t n, const void* dU3, const void* U3, const AdapterLists& l, bool f16, float* dA,
                          float* dB, cudaStream_t s) {
    static std::atomic<uint64_t> configured{0};
    if (!allow_smem(configured, (const void*)tc_adapter_grads, (int)kMaxSmem)) return QLORA_ERR_CUDA;
    GradParams p{};
    const int32_t RB = grad_block(r), Rg = grad_ranks(r);
    p.M = M; p.K = K; p.N = N; p.r = r; p.RB = RB;
    p.tiles_k = (int32_t)((K + 127) / 128);
    const int64_t tiles = p.tiles_k + (N + 127) / 128;
    if (tiles > INT32_MAX || n > 65535) return QLORA_ERR_SHAPE;
    p.v_bytes = (uint32_t)((3 * RB + 63) / 64) * 8192u;
    p.tmem_cols = RB <= 32 ? 128u : RB <= 64 ? 256u : 512u;
    // as many stages as fit in half of the shared memory (two CTAs per SM), else one CTA's worth
    uint32_t stages = (kMaxSmem / 2 - 3 * 1024) / (kStage16K + p.v_bytes);
    if (stages < 2) stages = (kMaxSmem - 3 * 1024) / (kStage16K + p.v_bytes);
    p.stages = std::min(stages, 4u);
    p.f16 = f16;
    p.n_grad = l.n_grad; p.e_grad = l.e_grad; p.tiles64 = l.tiles64;
    p.dA = dA; p.dB = dB;
    p.err = device_error_word();
    if (!p.err) return QLORA_ERR_CUDA;
    CUtensorMap tmX, tmdY, tmdU3, tmU3;
    if (!make_tmap_2d(&tmX, true, X, K, M, K * 2, 64, 64, true)) return QLORA_ERR_CUDA;
    if (!make_tmap_2d(&tmdY, true, dY, N, M, ldy * 2, 64, 64, true)) return QLORA_ERR_CUDA;
    if (!make_tmap_2d(&tmdU3, true, dU3, 3 * Rg, M, 6 * Rg, 64, 64, true)) return QLORA_ERR_CUDA;
    if (!make_tmap_2d(&tmU3, true, U3, 3 * Rg, M, 6 * Rg, 64, 64, true)) return QLORA_ERR_CUDA;
    const GradLayout lay = grad_layout(p.stages, p.v_bytes);
    (void)launch_dependent(tc_adapter_grads, dim3((unsigned)tiles, (unsigned)n, (unsigned)(Rg / RB)), dim3(kGradThreads),
                           lay.alloc, s, tmX, tmdY, tmdU3, tmU3, p);
    QLORA_CHECK_LAUNCH();
    return QLORA_OK;
}

// Checks that the entry points below share; n_adapters planes of B_all are rows of one tensor map.
qlora_status check_adapters(int64_t M, int64_t N, int64_t K, int32_t r, int32_t n) {
    QLORA_TRY(check_shape(N, K));
    QLORA_TRY(check_lora(M, r, 1.0f));
    if (n < 1 || n > 65535) return QLORA_ERR_INVALID_ARG;
    if (M > INT32_MAX - 512 || (int64_t)n * N > INT32_MAX - 512) return QLORA_ERR_SHAPE;
    return QLORA_OK;
}

// The fused GEMM of gemm_tc.cu over the tile lists: the forward (dx false) or dX.
qlora_status adapters_gemm(const qlora_nf4_weight* w, const void* A0, int64_t ld0, int64_t M, const void* V2, const void* B1,
                           int32_t b1_r, int32_t r, int32_t n, const AdapterLists& l, float* split_out, void* out,
                           int32_t out_dtype, bool dx, cudaStream_t s) {
    TcGemmArgs a{};
    a.w = w; a.A0 = A0; a.a0_ld = ld0; a.A1 = V2; a.B1 = B1; a.b1_r = b1_r; a.Rpad = half_width(r); a.n_adapters = n;
    a.split_out = split_out;
    a.p.M = M;
    a.p.Nout = dx ? w->K : w->N;
    a.p.ldo = a.p.Nout;
    a.p.out = out;
    a.p.out_f32 = out_dtype == QLORA_DTYPE_F32;
    a.p.ad.count = l.n512; a.p.ad.entry = l.e512; a.p.ad.cap = l.cap512;
    return launch_tc_gemm_nf4(a, dx, s);
}

}  // namespace
}  // namespace qlora

using namespace qlora;

extern "C" {

qlora_status qlora_adapters_workspace_size(int64_t M, int64_t N, int64_t K, int32_t r, int32_t n_adapters,
                                           size_t* bytes) {
    QLORA_TRY(check_adapters(M, N, K, r, n_adapters));
    if (!bytes) return QLORA_ERR_INVALID_ARG;
    *bytes = adapters_ws(M, N, K, r, n_adapters).total;
    return QLORA_OK;
}

qlora_status qlora_linear_fwd_adapters(const qlora_nf4_weight* w, const void* X, int64_t M, const void* A_all,
                                       const void* B_all, int32_t n_adapters, const int32_t* adapter_idx, int32_t r,
                                       const float* scales, void* Y, int32_t y_dtype, float* U_save, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    QLORA_TRY(check_weight(w));
    const int64_t N = w->N, K = w->K;
    QLORA_TRY(check_adapters(M, N, K, r, n_adapters));
    QLORA_TRY(check_dev(X));
    QLORA_TRY(check_dev(A_all));
    QLORA_TRY(check_dev(B_all));
    if (!adapter_idx || !scales) return QLORA_ERR_INVALID_ARG;
    if (!aligned_to(adapter_idx, 4) || !aligned_to(scales, 4)) return QLORA_ERR_ALIGN;
    QLORA_TRY(check_dev(Y));
    QLORA_TRY(check_out_dtype(y_dtype, w));
    if (U_save && !aligned16(U_save)) return QLORA_ERR_ALIGN;
    const AdaptersWs lw = adapters_ws(M, N, K, r, n_adapters);
    if (!workspace || workspace_bytes < lw.total) return QLORA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return QLORA_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = reinterpret_cast<char*>(align_up(reinterpret_cast<size_t>(workspace), 256));
    float* partial = reinterpret_cast<float*>(ws + lw.part);
    const bool f16 = w->compute_dtype == QLORA_DTYPE_F16;
    void* U2 = ws + lw.v2;
    const void* B8 = B_all;
    if (r % 8) {
        TimerScope t(QLORA_TIMER_LORA, s);
        QLORA_TRY(launch_pad_rows(B_all, n_adapters * N, r, ws + lw.b8, s));
        B8 = ws + lw.b8;
    }
    if (M <= kRowsMaxM) {
        RowsArgs a{};
        a.w = w; a.X = X; a.A = A_all; a.B = B8; a.ldb = round_up(r, 8); a.U2 = U2; a.R = half_width(r);
        a.idx = adapter_idx; a.scales = scales; a.n_adapters = n_adapters; a.r = r; a.M = M;
        a.out = Y; a.out_f32 = (y_dtype == QLORA_DTYPE_F32); a.U = U_save; a.workspace = ws + lw.part;
        TimerScope t(QLORA_TIMER_DECODE, s);
        return launch_rows(a, s);
    }
    const AdapterLists l = lists_at(ws, lw);
    {
        TimerScope t(QLORA_TIMER_LORA, s);
        QLORA_TRY(launch_lists(adapter_idx, M, n_adapters, lw, l, false, s));
        int splits = 0;
        QLORA_TRY(part_gemm(X, M, K, K, A_all, false, K, r, n_adapters, l, partial, f16, &splits, s));
        const FinishSource u{partial, splits, U_save, static_cast<uint16_t*>(U2), nullptr};
        QLORA_TRY(launch_finish(u, FinishSource{}, M, r, l, scales, f16, s));
    }
    TimerScope t(QLORA_TIMER_FWD_MAIN, s);
    return adapters_gemm(w, X, K, M, U2, B8, (int32_t)round_up(r, 8), r, n_adapters, l,
                         reinterpret_cast<float*>(ws + lw.split), Y, y_dtype, false, s);
}

qlora_status qlora_linear_bwd_adapters(const qlora_nf4_weight* w, const void* X, const void* dY, int64_t M,
                                       const void* A_all, const void* B_all, int32_t n_adapters,
                                       const int32_t* adapter_idx, int32_t r, const float* scales,
                                       const float* U_saved, void* dX, int32_t dx_dtype, float* dA_all, float* dB_all,
                                       void* workspace, size_t workspace_bytes, void* stream) {
    QLORA_TRY(check_weight(w));
    const int64_t N = w->N, K = w->K;
    QLORA_TRY(check_adapters(M, N, K, r, n_adapters));
    QLORA_TRY(check_dev(X));
    QLORA_TRY(check_dev(dY));
    QLORA_TRY(check_dev(A_all));
    QLORA_TRY(check_dev(B_all));
    if (!adapter_idx || !scales) return QLORA_ERR_INVALID_ARG;
    if (!aligned_to(adapter_idx, 4) || !aligned_to(scales, 4)) return QLORA_ERR_ALIGN;
    QLORA_TRY(check_dev(dA_all));
    QLORA_TRY(check_dev(dB_all));
    if (dX) {
        QLORA_TRY(check_dev(dX));
        QLORA_TRY(check_out_dtype(dx_dtype, w));
    }
    if (U_saved && !aligned16(U_saved)) return QLORA_ERR_ALIGN;
    const AdaptersWs lw = adapters_ws(M, N, K, r, n_adapters);
    if (!workspace || workspace_bytes < lw.total) return QLORA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return QLORA_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = reinterpret_cast<char*>(align_up(reinterpret_cast<size_t>(workspace), 256));
    float* partial = reinterpret_cast<float*>(ws + lw.part);
    const bool f16 = w->compute_dtype == QLORA_DTYPE_F16;
    const AdapterLists l = lists_at(ws, lw);
    uint16_t* dU2 = reinterpret_cast<uint16_t*>(ws + lw.v2);
    uint16_t* U3 = reinterpret_cast<uint16_t*>(ws + lw.u3);
    uint16_t* dU3 = reinterpret_cast<uint16_t*>(ws + lw.du3);
    const void* B8 = B_all;
    const void* dY8 = dY;
    const int64_t ldy = round_up(N, 8);
    {
        TimerScope t(QLORA_TIMER_LORA, s);
        QLORA_TRY(launch_lists(adapter_idx, M, n_adapters, lw, l, true, s));
        if (r % 8) {
            QLORA_TRY(launch_pad_rows(B_all, n_adapters * N, r, ws + lw.b8, s));
            B8 = ws + lw.b8;
        }
        if (N % 8) {
            QLORA_TRY(launch_pad_rows(dY, M, N, ws + lw.dy8, s));
            dY8 = ws + lw.dy8;
        }
        int splits = 0;
        if (!U_saved) {
            QLORA_TRY(part_gemm(X, M, K, K, A_all, false, K, r, n_adapters, l, partial, f16, &splits, s));
            const FinishSource u{partial, splits, nullptr, nullptr, U3};
            QLORA_TRY(launch_finish(u, FinishSource{}, M, r, l, scales, f16, s));
        }
        QLORA_TRY(part_gemm(dY8, M, N, ldy, B8, true, round_up(r, 8), r, n_adapters, l, partial, f16, &splits, s));
        const FinishSource du{partial, splits, nullptr, dX ? dU2 : nullptr, dU3};
        const FinishSource u{U_saved, 0, nullptr, nullptr, U_saved ? U3 : nullptr};
        QLORA_TRY(launch_finish(du, u, M, r, l, scales, f16, s));
    }
    // The adapter gradients run beside dX on the low-priority side stream and fill the SMs that its last
    // wave of tiles leaves idle.  Below about ten microseconds of dX the fork and join take longer on the
    // host than they save on the GPU, and the two run in turn.  So they do in a capture: the side stream is
    // one for all threads, and one thread's capture must not take in another's launches.
    bool forked = dX && (double)M * (double)N * (double)K >= 5e9;
    if (forked) {
        cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(s, &capture) != cudaSuccess) {
            (void)cudaGetLastError();
            return QLORA_ERR_CUDA;
        }
        forked = capture == cudaStreamCaptureStatusNone;
    }
    cudaStream_t g = forked ? side_stream() : s;
    cudaEvent_t join = nullptr;
    if (forked) {
        if (!g) return QLORA_ERR_CUDA;
        cudaEvent_t fork = nullptr;
        if (cudaEventCreateWithFlags(&fork, cudaEventDisableTiming) != cudaSuccess) return QLORA_ERR_CUDA;
        bool ok = cudaEventCreateWithFlags(&join, cudaEventDisableTiming) == cudaSuccess;
        ok = ok && cudaEventRecord(fork, s) == cudaSuccess && cudaStreamWaitEvent(g, fork, 0) == cudaSuccess;
        cudaEventDestroy(fork);
        if (!ok) {
            if (join) cudaEventDestroy(join);
            return QLORA_ERR_CUDA;
        }
    }
    qlora_status st = QLORA_OK;
    if (dX) {
        TimerScope t(QLORA_TIMER_DX_MAIN, s);
        st = adapters_gemm(w, dY8, ldy, M, dU2, A_all, r, r, n_adapters, l,
                           reinterpret_cast<float*>(ws + lw.split), dX, dx_dtype, true, s);
    }
    if (st == QLORA_OK) {
        TimerScope t(QLORA_TIMER_LORA, g);
        st = launch_grads(X, dY8, ldy, M, N, K, r, n_adapters, dU3, U3, l, f16, dA_all, dB_all, g);
    }
    if (forked) {   // the caller's stream resumes after the adapter gradients too
        const bool ok = cudaEventRecord(join, g) == cudaSuccess && cudaStreamWaitEvent(s, join, 0) == cudaSuccess;
        cudaEventDestroy(join);
        if (!ok && st == QLORA_OK) st = QLORA_ERR_CUDA;
    }
    return st;
}

}  // extern "C"
