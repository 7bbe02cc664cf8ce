// Distillation from a teacher's top logits: the loss that trains the adapters towards a 16-bit
// model's answers, of which only the k largest logits of each row are kept, and its gradient
// with respect to the student's logits (the dY of the output projection's backward).
//
// For row m with valid entries j (0 <= i_j < V), teacher logits t_j and student logits z:
//     p_j   = exp(t_j/T) / sum over the valid entries         (softmax over the kept logits)
//     lse   = log sum_v exp(z_v/T)                            (over the whole vocabulary)
//     loss  = T^2 sum_j p_j (log p_j - (z_{i_j}/T - lse))     (KL divergence, scaled by T^2)
//     dz_v  = dloss T (exp(z_v/T - lse) - sum_{j: i_j = v} p_j)
// A row without valid entries (none given, or every t_j = -inf) has loss 0 and gradient 0, and so has a row
// whose logits are all masked (masked_from below): its lse is -inf.
//
// Both kernels are bound by HBM: the forward reads every logit once (running maximum and sum of
// the softmax in registers, fp32, base-2 exponentials), the backward reads and writes every
// element once.  A row is a CTA's work; when there are too few rows to fill the GPU, the forward
// gives a row to a cluster of up to 8 CTAs that join their (maximum, sum) pairs through
// distributed shared memory, and the backward cuts the row into independent parts (the saved lse
// is all that a part needs of the others).
#include <climits>
#include <cmath>

#include <cooperative_groups.h>

#include "qlora_internal.cuh"

namespace cg = cooperative_groups;

namespace qlora {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = 1024;                     // teacher entries per row
constexpr int kTopPerThread = kMaxTop / kThreads;
constexpr float kLn2 = 0.6931471805599453f;
constexpr double kLog2e = 1.4426950408889634;

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two additions in one instruction, each rounded as __fadd_rn.
__device__ __forceinline__ float2 add2_rn(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

template <int DT>
__device__ __forceinline__ float load1(const void* base, int64_t e) {
    if constexpr (DT == QLORA_DTYPE_F32) return static_cast<const float*>(base)[e];
    else return from16(static_cast<const uint16_t*>(base)[e], DT == QLORA_DTYPE_F16);
}

__device__ __forceinline__ float load_any(const void* base, int64_t e, int dt) {
    return dt == QLORA_DTYPE_F32 ? static_cast<const float*>(base)[e]
                                 : from16(static_cast<const uint16_t*>(base)[e], dt == QLORA_DTYPE_F16);
}

template <int DT>
__device__ __forceinline__ void store1(void* base, int64_t e, float v) {
    if constexpr (DT == QLORA_DTYPE_F32) static_cast<float*>(base)[e] = v;
    else static_cast<uint16_t*>(base)[e] = (uint16_t)to16_rn(v, DT == QLORA_DTYPE_F16);
}

// Eight consecutive elements as loaded, in one access that is aligned to its size (16 bytes of a 16-bit type,
// 32 of fp32: a warp's two halves of 16 bytes would each touch every sector).
template <int DT>
struct Raw8 {
    uint4 a, b;
    __device__ __forceinline__ void load(const void* base, int64_t e) {
        if constexpr (DT == QLORA_DTYPE_F32) {
            asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                         : "l"(static_cast<const float*>(base) + e));
        } else {
            a = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + e));
        }
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        if constexpr (DT == QLORA_DTYPE_F32) {
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
        } else {
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DT == QLORA_DTYPE_F16) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                    v[2 * i] = f.x;
                    v[2 * i + 1] = f.y;
                } else {
                    v[2 * i] = __uint_as_float(w[i] << 16);
                    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
                }
            }
        }
    }
};

template <int DT>
__device__ __forceinline__ void store8(void* base, int64_t e, const float (&v)[8]) {
    if constexpr (DT == QLORA_DTYPE_F32) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
        store_sector(static_cast<float*>(base) + e, w);
    } else {
        constexpr bool h = DT == QLORA_DTYPE_F16;
        __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + e),
               make_uint4(pack16x2_rn(v[0], v[1], h), pack16x2_rn(v[2], v[3], h), pack16x2_rn(v[4], v[5], h),
                          pack16x2_rn(v[6], v[7], h)));
    }
}

// Running maximum and sum of exponentials: sum_i exp(x_i / T) = s 2^(ref(m) c), c = log2(e) / T.  The
// difference to the maximum is taken before the scaling, so that the largest logit contributes exactly 1 and no
// exponent is above 0, for logits of any size: with fma(x, c, -r) and r the rounded m c, what r's rounding
// leaves over exceeds 128 for masks such as -1e10, and a thread of masks only has s = inf.
// m = -inf stands for an empty sum; the reference is 0 then, so -inf logits add zeros and never meet
// -inf - -inf.  So it is for +inf, of which s then is.
struct Softmax2 {
    float m, s;
    __device__ __forceinline__ static float ref(float m) { return fabsf(m) == INFINITY ? 0.f : m; }
    __device__ __forceinline__ static float term(float x, float r, float c) {
        return exp2_approx(__fmul_rn(__fsub_rn(x, r), c));
    }
    // PAIRS: differences and products two at a time, the same values.  For logits of 16 bits (a call at
    // [4096, 128000] bf16: 186.2 us, one by one 188.5); fp32 logits leave no registers for it (the kernel at
    // [1023, 50001]: 41.2 us in pairs, 38.8 one by one).
    template <bool PAIRS, int N>
    __device__ __forceinline__ void add(const float (&x)[N], float c) {
        float mn = fmaxf(m, x[0]);
#pragma unroll
        for (int i = 1; i < N; ++i) mn = fmaxf(mn, x[i]);
        const float r = ref(mn);
        float acc0 = 0.f, acc1 = 0.f;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            if constexpr (PAIRS) {
                const float2 y = mul2_rn(add2_rn(make_float2(x[i], x[i + 1]), make_float2(-r, -r)), make_float2(c, c));
                acc0 += exp2_approx(y.x);
                acc1 += exp2_approx(y.y);
            } else {
                acc0 += term(x[i], r, c);
                if (i + 1 < N) acc1 += term(x[i + 1], r, c);
            }
        }
        s = __fmaf_rn(s, term(m, r, c), acc0 + acc1);
        m = mn;
    }
    __device__ __forceinline__ void join(float m2, float s2, float c) {
        const float mn = fmaxf(m, m2), r = ref(mn);
        s = s * term(m, r, c) + s2 * term(m2, r, c);
        m = mn;
    }
};

// A row whose largest logit is not above this is masked throughout: the type's lowest value in fp16, and -1e8
// in bf16 and fp32, far from any logit of a model, where one fp32 lse cannot hold log V beside the mask
// (masks of -1e9, -1e10, -1e30, the lowest value).
template <int DT>
constexpr float masked_from() { return DT == QLORA_DTYPE_F16 ? -65504.f : -1e8f; }

struct DistillParams {
    const void* logits;       // [M, V], rows ld elements apart
    int64_t ld;
    int64_t M, V;
    const int32_t* idx;       // [M, k]
    const void* t;            // [M, k]
    int32_t t_dtype, k;
    float c;                  // log2(e) / T
    float T;
    float* loss;              // [M]            (forward)
    float* lse;               // [M]            (written by the forward, read by the backward)
    const float* dloss;       // [M]            (backward)
    void* dlogits;            // [M, V], rows ldd elements apart
    int64_t ldd;
    int32_t parts;            // CTAs of a row
    uint32_t* err;
};

// A row's teacher entries in shared memory: index (-1: no entry) and teacher logit (-inf: no entry); the
// student's logits there are in registers of the thread that loaded the entry, e = tid + 256 q, so that
// nothing waits for them before their use.  An index outside [0, V) is no entry; one at or above V raises the BOUNDS flag.
struct Entries {
    int32_t i[kMaxTop];
    float t[kMaxTop];
};

// Fills the entries of row m; z only where the element lies in [lo, hi) or [0, head).  Returns whether
// the calling thread met an entry that is not -inf.
template <int DT_IN>
__device__ __forceinline__ bool load_entries(const DistillParams& p, int64_t m, const void* row, int64_t lo, int64_t hi,
                                             int64_t head, Entries& s, float (&z)[kTopPerThread]) {
    bool any = false;
#pragma unroll
    for (int q = 0; q < kTopPerThread; ++q) {
        const int e = threadIdx.x + q * kThreads;
        z[q] = 0.f;
        if (e >= p.k) continue;
        int32_t i = p.idx[m * p.k + e];
        if (i >= p.V) atomicOr(p.err, ERR_FLAG_BOUNDS);
        if (i < 0 || i >= p.V) i = -1;
        const float t = i >= 0 ? load_any(p.t, m * p.k + e, p.t_dtype) : -INFINITY;
        if (i >= 0 && ((i >= lo && i < hi) || i < head)) z[q] = load1<DT_IN>(row, i);
        s.i[e] = i;
        s.t[e] = t;
        any |= !(t == -INFINITY);
    }
    return any;
}

// The teacher's softmax over the entries, by one warp: log2 p_e = (t_e - ref) c - l.  The differences to
// the row's largest logit are taken before the scaling, so rows of the type's lowest value stay finite.
// The maximum skips NaN and the sum does not: a NaN among the row's teacher logits gives NaN.
struct Teacher {
    float ref, l;
    bool some;                 // the row has an entry
};
__device__ __forceinline__ Teacher teacher_softmax(const Entries& s, int k, float c) {
    const int lane = threadIdx.x & 31;
    float mx = -INFINITY, sum = 0.f;
    for (int e = lane; e < k; e += 32) mx = fmaxf(mx, s.t[e]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float ref = Softmax2::ref(mx);
    for (int e = lane; e < k; e += 32) sum += exp2f(__fmul_rn(__fsub_rn(s.t[e], ref), c));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return Teacher{ref, log2f(sum), !(sum == 0.f)};
}
__device__ __forceinline__ float log2_p(const Teacher& t, float logit, float c) {
    return __fsub_rn(__fmul_rn(__fsub_rn(logit, t.ref), c), t.l);
}

// Row layout of a part: elements [0, head) one by one, then chunks of eight from `head` on, then
// the tail one by one; head brings the chunks to multiples of their size.
template <int DT_IN>
__global__ void __launch_bounds__(kThreads, 5) distill_fwd(DistillParams p) {
    grid_dependency_wait();
    allow_dependents();
    __shared__ Entries entries;
    __shared__ float entry_z[kMaxTop];
    __shared__ float2 joined[8];
    const int part = (int)(blockIdx.x % (unsigned)p.parts);
    const int64_t m = blockIdx.x / (unsigned)p.parts;
    constexpr int kEs = DT_IN == QLORA_DTYPE_F32 ? 4 : 2;
    const char* row = static_cast<const char*>(p.logits) + m * p.ld * kEs;

    // a cluster's CTAs have all started before one writes another's shared memory
    if (p.parts > 1) cg::this_cluster().barrier_arrive();
    float z[kTopPerThread];
    if (part == 0) (void)load_entries<DT_IN>(p, m, row, 0, p.V, 0, entries, z);

    const int64_t head = min(p.V, (int64_t)(-(int64_t)(reinterpret_cast<uintptr_t>(row) / kEs) & 7));
    const int64_t chunks = (p.V - head) / 8;
    const int64_t c0 = chunks * part / p.parts, c1 = chunks * (part + 1) / p.parts;
    Softmax2 acc{-INFINITY, 0.f};
    constexpr int kUnroll = DT_IN == QLORA_DTYPE_F32 ? 3 : 6; // bytes in flight per thread: 96, 166.6 us; 64, 172 ([4096, 128000] bf16)
    int64_t c = c0 + threadIdx.x;
    for (; c + (kUnroll - 1) * kThreads < c1; c += kUnroll * kThreads) {
        Raw8<DT_IN> raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) raw[u].load(row, head + 8 * (c + u * kThreads));
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float v[8];
            raw[u].values(v);
            acc.add<DT_IN != QLORA_DTYPE_F32>(v, p.c);
        }
    }
    for (; c < c1; c += kThreads) {
        Raw8<DT_IN> raw;
        raw.load(row, head + 8 * c);
        float v[8];
        raw.values(v);
        acc.add<DT_IN != QLORA_DTYPE_F32>(v, p.c);
    }
    if (part == p.parts - 1) {                                // fewer than 8 + 8 single elements
        const int64_t tail0 = head + 8 * chunks, singles = head + (p.V - tail0);
        if (threadIdx.x < singles) {
            const float v[1] = {load1<DT_IN>(row, threadIdx.x < head ? threadIdx.x : tail0 + (threadIdx.x - head))};
            acc.add<false>(v, p.c);
        }
    }

#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, acc.m, o), s2 = __shfl_xor_sync(0xffffffffu, acc.s, o);
        acc.join(m2, s2, p.c);
    }
    __shared__ float2 warp_acc[kWarps];
    if (part == 0)
#pragma unroll
        for (int q = 0; q < kTopPerThread; ++q)
            if ((int)threadIdx.x + q * kThreads < p.k) entry_z[threadIdx.x + q * kThreads] = z[q];
    if ((threadIdx.x & 31) == 0) warp_acc[threadIdx.x >> 5] = make_float2(acc.m, acc.s);
    __syncthreads();
    acc = Softmax2{warp_acc[0].x, warp_acc[0].y};
#pragma unroll
    for (int w = 1; w < kWarps; ++w) acc.join(warp_acc[w].x, warp_acc[w].y, p.c);
    if (p.parts > 1) {                                        // the row's CTAs are one cluster
        cg::cluster_group cluster = cg::this_cluster();
        cluster.barrier_wait();
        if (threadIdx.x == 0) *cluster.map_shared_rank(&joined[part], 0) = make_float2(acc.m, acc.s);
        cluster.sync();
        if (part != 0) return;
        acc = Softmax2{joined[0].x, joined[0].y};
        for (int w = 1; w < p.parts; ++w) acc.join(joined[w].x, joined[w].y, p.c);
    }
    if (threadIdx.x >= 32) return;                            // one warp ends the row
    // loss = T sum_e p_e (T (log p_e + log s) - (z_e - ref)): logits only as differences, which the temperature
    // does not scale up, so that a masked z_e costs its distance and not inf
    const float ref = Softmax2::ref(acc.m), log_s = log2f(acc.s) * kLn2;
    const Teacher teacher = teacher_softmax(entries, p.k, p.c);
    float sum = 0.f;
    for (int e = threadIdx.x; e < p.k; e += 32) {
        const float lp = log2_p(teacher, entries.t[e], p.c), pe = exp2f(lp);
        if (entries.i[e] >= 0 && !(pe == 0.f))
            sum += pe * __fsub_rn(__fmul_rn(__fmaf_rn(lp, kLn2, log_s), p.T), __fsub_rn(entry_z[e], ref));
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const bool masked = acc.m <= masked_from<DT_IN>() && acc.s == acc.s;   // a NaN, which the maximum skips, is in s
    if (threadIdx.x == 0) {
        p.lse[m] = masked ? -INFINITY : __fdiv_rn(ref, p.T) + log_s;
        p.loss[m] = teacher.some && !masked ? p.T * sum : 0.f;
    }
}

template <int DT_IN, int DT_OUT, bool VEC>
__global__ void __launch_bounds__(kThreads, DT_IN != QLORA_DTYPE_F32 && DT_OUT != QLORA_DTYPE_F32 ? 5 : 4)
distill_bwd(DistillParams p) {
    grid_dependency_wait();
    allow_dependents();
    __shared__ Entries entries;
    const int part = (int)(blockIdx.x % (unsigned)p.parts);
    // the rows run from the last to the first: what the forward has read last is still in L2
    const int64_t m = p.M - 1 - blockIdx.x / (unsigned)p.parts;
    constexpr int kEs = DT_IN == QLORA_DTYPE_F32 ? 4 : 2, kEd = DT_OUT == QLORA_DTYPE_F32 ? 4 : 2;
    const char* row = static_cast<const char*>(p.logits) + m * p.ld * kEs;
    char* drow = static_cast<char*>(p.dlogits) + m * p.ldd * kEd;
    // VEC: chunks of eight are aligned to their size in both rows, from element `head` on
    const int64_t head = VEC ? min(p.V, (int64_t)(-(int64_t)(reinterpret_cast<uintptr_t>(row) / kEs) & 7)) : 0;
    const int64_t chunks = VEC ? (p.V - head) / 8 : 0;
    const int64_t c0 = chunks * part / p.parts, c1 = chunks * (part + 1) / p.parts;
    const bool last = part == p.parts - 1;
    // this part's elements: [lo, hi), and the last part's head [0, head) and tail too
    const int64_t lo = VEC ? head + 8 * c0 : p.V * part / p.parts;
    const int64_t hi = VEC ? (last ? p.V : head + 8 * c1) : p.V * (part + 1) / p.parts;

    // Only what the dense pass must wait for comes before it: whether the row has an entry, and the
    // entries' logits of this part, which it may overwrite (the gradient may take the logits' place).  The
    // teacher's softmax follows the pass.
    const float g = p.dloss[m], scale = g * p.T, lse = p.lse[m], l2 = __fmul_rn(lse, (float)kLog2e);
    float z[kTopPerThread];
    const bool entry = load_entries<DT_IN>(p, m, row, lo, hi, last ? head : 0, entries, z);
    const bool zero = !__syncthreads_or(entry) || g == 0.f || lse == -INFINITY;

    if (VEC) {
        // measured best of 2 to 8 loads per thread, and of 3 to 8 blocks per SM
        constexpr int kUnroll = DT_IN == QLORA_DTYPE_F32 ? 3 : 4;
        int64_t c = c0 + threadIdx.x;
        if (zero) {
            const float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            for (; c < c1; c += kThreads) store8<DT_OUT>(drow, head + 8 * c, v);
        } else {
            for (; c + (kUnroll - 1) * kThreads < c1; c += kUnroll * kThreads) {
                Raw8<DT_IN> raw[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) raw[u].load(row, head + 8 * (c + u * kThreads));
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    float v[8];
                    raw[u].values(v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = scale * exp2_approx(__fmaf_rn(v[i], p.c, -l2));
                    store8<DT_OUT>(drow, head + 8 * (c + u * kThreads), v);
                }
            }
            for (; c < c1; c += kThreads) {
                Raw8<DT_IN> raw;
                raw.load(row, head + 8 * c);
                float v[8];
                raw.values(v);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = scale * exp2_approx(__fmaf_rn(v[i], p.c, -l2));
                store8<DT_OUT>(drow, head + 8 * c, v);
            }
        }
        if (last) {
            const int64_t tail0 = head + 8 * chunks, singles = head + (p.V - tail0), tid = threadIdx.x;
            if (tid < singles) {
                const int64_t e = tid < head ? tid : tail0 + (tid - head);
                store1<DT_OUT>(drow, e, zero ? 0.f : scale * exp2_approx(__fmaf_rn(load1<DT_IN>(row, e), p.c, -l2)));
            }
        }
    } else {
        for (int64_t e = lo + threadIdx.x; e < hi; e += kThreads)
            store1<DT_OUT>(drow, e, zero ? 0.f : scale * exp2_approx(__fmaf_rn(load1<DT_IN>(row, e), p.c, -l2)));
    }
    if (zero) return;

    // the entries' elements: the first of equal indices carries the sum of their probabilities
    const Teacher teacher = teacher_softmax(entries, p.k, p.c);   // every warp for itself
    __syncthreads();                                          // every warp has read the entries
#pragma unroll
    for (int q = 0; q < kTopPerThread; ++q) {
        const int e = threadIdx.x + q * kThreads;
        if (e < p.k) entries.t[e] = exp2f(log2_p(teacher, entries.t[e], p.c));
    }
    __syncthreads();                                          // the dense pass has been written, too
#pragma unroll
    for (int q = 0; q < kTopPerThread; ++q) {
        const int e = threadIdx.x + q * kThreads;
        const int32_t i = e < p.k ? entries.i[e] : -1;
        if (i < 0 || !((i >= lo && i < hi) || (last && i < head))) continue;
        float sum = 0.f;
        bool first = true;
        for (int o = 0; o < p.k; ++o) {
            if (entries.i[o] != i) continue;
            first &= o >= e;
            sum += entries.t[o];
        }
        if (first) store1<DT_OUT>(drow, i, scale * (exp2_approx(__fmaf_rn(z[q], p.c, -l2)) - sum));
    }
}

inline int elem_size(int dt) { return dt == QLORA_DTYPE_F32 ? 4 : 2; }

// CTAs of a row: enough to give every SM two, in powers of two up to a portable cluster's eight,
// while each still has 4096 elements (two passes of the block).
int row_parts(int64_t M, int64_t V) {
    int parts = 1;
    while (parts < 8 && M * parts < 2 * 148 && V / (2 * parts) >= 4096) parts *= 2;
    return parts;
}

template <int DT_IN>
cudaError_t run_fwd(const DistillParams& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.M * p.parts));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, distill_fwd<DT_IN>, p);
}

template <int DT_IN, int DT_OUT>
cudaError_t run_bwd2(const DistillParams& p, cudaStream_t s) {
    const dim3 grid((unsigned)(p.M * p.parts));
    // chunks of eight are aligned in both rows when the rows' first elements lie alike modulo eight
    constexpr int64_t kEs = DT_IN == QLORA_DTYPE_F32 ? 4 : 2, kEd = DT_OUT == QLORA_DTYPE_F32 ? 4 : 2;
    const int64_t z0 = (int64_t)(reinterpret_cast<uintptr_t>(p.logits) / kEs & 7);
    const int64_t d0 = (int64_t)(reinterpret_cast<uintptr_t>(p.dlogits) / kEd & 7);
    if (z0 == d0 && (p.ld - p.ldd) % 8 == 0)
        return launch_dependent(distill_bwd<DT_IN, DT_OUT, true>, grid, dim3(kThreads), 0, s, p);
    return launch_dependent(distill_bwd<DT_IN, DT_OUT, false>, grid, dim3(kThreads), 0, s, p);
}

template <int DT_IN>
cudaError_t run_bwd(const DistillParams& p, int d_dtype, cudaStream_t s) {
    if (d_dtype == QLORA_DTYPE_F32) return run_bwd2<DT_IN, QLORA_DTYPE_F32>(p, s);
    if (d_dtype == QLORA_DTYPE_F16) return run_bwd2<DT_IN, QLORA_DTYPE_F16>(p, s);
    return run_bwd2<DT_IN, QLORA_DTYPE_BF16>(p, s);
}

// A device pointer of elements of `bytes` bytes: present and aligned to them.
qlora_status check_elems(const void* p, int bytes) {
    if (!p) return QLORA_ERR_INVALID_ARG;
    return aligned_to(p, (uintptr_t)bytes) ? QLORA_OK : QLORA_ERR_ALIGN;
}

bool dtype_ok(int32_t dt) { return dt == QLORA_DTYPE_BF16 || dt == QLORA_DTYPE_F16 || dt == QLORA_DTYPE_F32; }

// The checks that both directions share; fills the common parameters.
qlora_status distill_args(const void* logits, int32_t z_dtype, int64_t ld, int64_t M, int64_t V, const int32_t* idx,
                          const void* t, int32_t t_dtype, int32_t k, float T, DistillParams& p) {
    if (!dtype_ok(z_dtype) || !dtype_ok(t_dtype)) return QLORA_ERR_INVALID_ARG;
    QLORA_TRY(check_elems(logits, elem_size(z_dtype)));
    QLORA_TRY(check_elems(idx, 4));
    QLORA_TRY(check_elems(t, elem_size(t_dtype)));
    if (k < 1 || k > kMaxTop) return QLORA_ERR_INVALID_ARG;
    // log2(e) / T and T^2 keep their digits and the products with logits their range within these limits
    if (!(T >= 1e-3f && T <= 1e3f)) return QLORA_ERR_INVALID_ARG;
    if (M < 1 || V < 1 || V > INT32_MAX || ld < V || M > INT32_MAX / 8 || ld > (int64_t(1) << 40) / M)
        return QLORA_ERR_SHAPE;
    p.logits = logits; p.ld = ld; p.M = M; p.V = V;
    p.idx = idx; p.t = t; p.t_dtype = t_dtype; p.k = k;
    p.c = (float)(kLog2e / (double)T); p.T = T;
    p.parts = row_parts(M, V);
    return QLORA_OK;
}

}  // namespace
}  // namespace qlora

using namespace qlora;

extern "C" {

qlora_status qlora_distill_topk_fwd(const void* logits, int32_t z_dtype, int64_t ld, int64_t M, int64_t V,
                                    const int32_t* teacher_idx, const void* teacher_logits, int32_t t_dtype, int32_t k,
                                    float temperature, float* loss, float* lse, void* stream) {
    DistillParams p{};
    QLORA_TRY(distill_args(logits, z_dtype, ld, M, V, teacher_idx, teacher_logits, t_dtype, k, temperature, p));
    QLORA_TRY(check_elems(loss, 4));
    QLORA_TRY(check_elems(lse, 4));
    p.loss = loss; p.lse = lse;
    p.err = device_error_word();
    if (!p.err) return QLORA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (z_dtype == QLORA_DTYPE_F32) (void)run_fwd<QLORA_DTYPE_F32>(p, s);
    else if (z_dtype == QLORA_DTYPE_F16) (void)run_fwd<QLORA_DTYPE_F16>(p, s);
    else (void)run_fwd<QLORA_DTYPE_BF16>(p, s);
    QLORA_CHECK_LAUNCH();
    return QLORA_OK;
}

qlora_status qlora_distill_topk_bwd(const void* logits, int32_t z_dtype, int64_t ld, int64_t M, int64_t V,
                                    const int32_t* teacher_idx, const void* teacher_logits, int32_t t_dtype, int32_t k,
                                    float temperature, const float* lse, const float* dloss, void* dlogits,
                                    int32_t d_dtype, int64_t ldd, void* stream) {
    DistillParams p{};
    QLORA_TRY(distill_args(logits, z_dtype, ld, M, V, teacher_idx, teacher_logits, t_dtype, k, temperature, p));
    if (!dtype_ok(d_dtype)) return QLORA_ERR_INVALID_ARG;
    QLORA_TRY(check_elems(lse, 4));
    QLORA_TRY(check_elems(dloss, 4));
    QLORA_TRY(check_elems(dlogits, elem_size(d_dtype)));
    if (ldd < V || ldd > (int64_t(1) << 40) / M) return QLORA_ERR_SHAPE;
    // in place (the same rows of the same type) or apart: anything between would read written values
    const uintptr_t z0 = reinterpret_cast<uintptr_t>(logits), d0 = reinterpret_cast<uintptr_t>(dlogits);
    const uintptr_t z1 = z0 + (uintptr_t)((M - 1) * ld + V) * elem_size(z_dtype);
    const uintptr_t d1 = d0 + (uintptr_t)((M - 1) * ldd + V) * elem_size(d_dtype);
    const bool same = z0 == d0 && ld == ldd && elem_size(z_dtype) == elem_size(d_dtype);
    if (!same && z0 < d1 && d0 < z1) return QLORA_ERR_INVALID_ARG;
    p.lse = const_cast<float*>(lse); p.dloss = dloss; p.dlogits = dlogits; p.ldd = ldd;
    p.err = device_error_word();
    if (!p.err) return QLORA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (z_dtype == QLORA_DTYPE_F32) (void)run_bwd<QLORA_DTYPE_F32>(p, d_dtype, s);
    else if (z_dtype == QLORA_DTYPE_F16) (void)run_bwd<QLORA_DTYPE_F16>(p, d_dtype, s);
    else (void)run_bwd<QLORA_DTYPE_BF16>(p, d_dtype, s);
    QLORA_CHECK_LAUNCH();
    return QLORA_OK;
}

}  // extern "C"
