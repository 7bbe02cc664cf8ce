// What the fused dequant-GEMMs share: the expansion of packed 4-bit codes to the 16-bit compute type by
// their producer warps (a 16-entry table per block of 64 weights held in registers, and byte permutes)
// and the output stores of their epilogues.
#pragma once

#include "qlora_internal.cuh"

namespace qlora {

// prmt.b32 in its default mode: byte i of the result is source byte (s_i & 7)
// of {y, x}; when bit 3 of the selector nibble s_i is set, that byte's sign bit
// is replicated over all 8 bits.  (The __byte_perm intrinsic ignores bit 3, so
// the sign-replicating selectors below need the instruction itself.)
__device__ __forceinline__ uint32_t prmt(uint32_t x, uint32_t y, uint32_t s) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(s));
    return r;
}

struct Lut {
    uint32_t L[4], H[4];   // low / high bytes of the 16 bf16 entries, 4 entries per register
};

__device__ __forceinline__ void build_lut(Lut& t, float c1p, const NF4Tables& tb, bool f16) {
    uint32_t P[8];   // entries 2j, 2j+1 rounded to the compute dtype (bf16 or fp16), packed
    const float2 c2p = make_float2(c1p, c1p);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 e = mul2_rn(make_float2(tb.q[2 * j], tb.q[2 * j + 1]), c2p);   // fp32(q * c1'), per element
        P[j] = pack16x2_rn(e.x, e.y, f16);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        t.L[j] = prmt(P[2 * j], P[2 * j + 1], 0x6420);
        t.H[j] = prmt(P[2 * j], P[2 * j + 1], 0x7531);
    }
}

// 8 codes (4 packed bytes, element 2j in the high nibble of byte j) -> 8 bf16.
// The nibbles of w run e1, e0, e3, e2, ... from the least significant end; the
// table permutes keep that pair-swapped order and the final interleave undoes
// it.  Bytes whose code is >= 8 take entries 8-15 (sign-replicated bit 3).
__device__ __forceinline__ uint4 expand8(uint32_t w, const Lut& t) {
    const uint32_t u = w << 4;             // bit 3 of the low nibble of each byte -> that byte's bit 7
    const uint32_t wm = w & 0x77777777u;   // table index of every code; prmt reads selector bits 0-15
    uint32_t o[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t sel = h == 0 ? wm : (wm >> 16);
        const uint32_t mask = prmt(u, w, h == 0 ? 0xD9C8u : 0xFBEAu);
        const uint32_t la = prmt(t.L[0], t.L[1], sel);
        const uint32_t lb = prmt(t.L[2], t.L[3], sel);
        const uint32_t ha = prmt(t.H[0], t.H[1], sel);
        const uint32_t hb = prmt(t.H[2], t.H[3], sel);
        const uint32_t lo = (la & ~mask) | (lb & mask);
        const uint32_t hi = (ha & ~mask) | (hb & mask);
        o[2 * h] = prmt(lo, hi, 0x4051);
        o[2 * h + 1] = prmt(lo, hi, 0x6273);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr)
                 : "memory");
    return v;
}

// Expand one NF4 block (64 weights of one W row) into one 128-byte swizzled
// row of a B image.  code_lo/code_hi: the two 16-byte halves of its codes.
__device__ __forceinline__ void expand_block_row(uint32_t row_addr, uint32_t row_in_atom, uint4 c0, uint4 c1,
                                                 const Lut& t) {
    const uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
    for (int c = 0; c < 8; ++c) st_shared_v4(row_addr + ((c ^ row_in_atom) << 4), expand8(w[c], t));
}

__device__ __forceinline__ void zero_row(uint32_t row_addr) {
#pragma unroll
    for (int c = 0; c < 8; ++c) st_shared_v4(row_addr + (c << 4), make_uint4(0, 0, 0, 0));
}

// The same row in a non-swizzled K-major image (rows 16 bytes apart, chunk c of
// every row LBO bytes after chunk 0): the eight stores take immediate offsets from
// one address, and a warp's 32 rows fill 512 contiguous bytes per chunk.
template <uint32_t LBO>
__device__ __forceinline__ void expand_block_row_kn(uint32_t row_addr, uint4 c0, uint4 c1, const Lut& t) {
    const uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
    for (int c = 0; c < 8; ++c) st_shared_v4(row_addr + c * LBO, expand8(w[c], t));
}

template <uint32_t LBO>
__device__ __forceinline__ void zero_row_kn(uint32_t row_addr) {
#pragma unroll
    for (int c = 0; c < 8; ++c) st_shared_v4(row_addr + c * LBO, make_uint4(0, 0, 0, 0));
}

// Store 32 consecutive output columns nb .. nb+31 of row m (fp32, or rounded to the 16-bit
// compute dtype); columns at or past nlim (the end of the tile or of the row) are skipped.
__device__ __forceinline__ void store_row32(void* out, bool out_f32, bool h, int64_t ldo, int64_t m, int64_t nb,
                                            int64_t nlim, const uint32_t (&v)[32]) {
    const bool full = (nb + 32 <= nlim);
    if (out_f32) {
        float* dst = static_cast<float*>(out) + m * ldo + nb;
        if (full && (reinterpret_cast<uintptr_t>(dst) & 31u) == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) store_sector(dst + 8 * i, v + 8 * i);
        } else if (full && (ldo & 3) == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                reinterpret_cast<uint4*>(dst)[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (nb + i < nlim) dst[i] = __uint_as_float(v[i]);
        }
    } else {
        uint16_t* dst = static_cast<uint16_t*>(out) + m * ldo + nb;
        if (full && (ldo & 7) == 0) {
            uint32_t o[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = pack16x2_rn(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), h);
            if ((reinterpret_cast<uintptr_t>(dst) & 31u) == 0) {
                store_sector(dst, o);
                store_sector(dst + 16, o + 8);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    reinterpret_cast<uint4*>(dst)[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (nb + i < nlim) dst[i] = (uint16_t)to16_rn(__uint_as_float(v[i]), h);
        }
    }
}

}  // namespace qlora
