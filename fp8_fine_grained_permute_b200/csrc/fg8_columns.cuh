// fg8_columns.cuh -- pieces of the kernels that quantize fp32 values or read 8-bit
// rows: tile scales, code conversions, and the tiles of the token axis.
#pragma once

#include <cuda_fp16.h>

#include "fg8_common.cuh"

namespace fg8 {

constexpr int kColsMaxE = 1024;

// Two E4M3 codes in shared memory -> fp32.  A 16-bit load hands the conversion its
// operand as it is; taking a word apart costs two instructions of the pipe (ALU,
// with the conversions, maxima and byte permutes) that bounds these kernels.
FG8_DEV float2 e4m3x2_at(uint32_t addr) {
    uint32_t h;
    asm volatile(
        "{\n"
        ".reg .b16 c;\n"
        "ld.shared.b16 c, [%1];\n"
        "cvt.rn.f16x2.e4m3x2 %0, c;\n"
        "}\n"
        : "=r"(h)
        : "r"(addr)
        : "memory");
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// tile_scale for tiles of fp32 values: where amax / 448 rounds to 0 (amax below
// 2^-141, which no tile of 16-bit values reaches) the scale is the smallest
// positive number, so that no code is a quotient by 0.
FG8_DEV float tile_scale32(float amax) {
    const float s = tile_scale(amax);
    return s == 0.0f ? 1.4e-45f : s;
}

// The scale of a tile of fp32 values without the division routine: q = amax /
// 448 from the rounded reciprocal and one residual correction, the IEEE quotient
// for every amax >= 2^-110 (tests/test_corrected_quotient.py); below that the division.
FG8_DEV float tile_scale_fast(float amax) {
    if (amax < 0x1p-110f) return tile_scale32(amax);
    const float r = 1.0f / 448.0f;
    const float q = __fmul_rn(amax, r);
    return __fmaf_rn(__fmaf_rn(-q, 448.0f, amax), r, q);
}

// A code factor for scale s: E4M3(x * inv_scale(s)) is x / s rounded with a
// relative error of 2^-22 before the rounding to 4 bits.  Subnormal scales
// (amax < 448 * 2^-126) have no finite fp32 reciprocal: callers divide there.
FG8_DEV float inv_scale(float s) {
    float r0;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r0) : "f"(s));
    return __fmaf_rn(r0, __fmaf_rn(-s, r0, 1.0f), r0);
}
FG8_DEV bool scale_subnormal(float s) { return !(s >= 1.17549435e-38f); }

// The code of a quotient x / s without a division: with r = fp32(1 / s) correctly
// rounded, z0 = fp32(x r) and z = fp32(z0 + fp32(x - z0 s) r), z is the quotient to
// 2^-46 before its own rounding, so it can differ from the IEEE quotient (by one fp32
// step) only where x / s lies that close to the middle of two fp32 numbers.  E4M3(z)
// and E4M3(fp32(x / s)) differ only if those two numbers are a rounding border of
// E4M3 (a value of at most 5 significant bits) and its neighbour; that leaves the
// significands of s within 8 units of a multiple of 2^20 and, for each border, a
// handful of x, and for every one of these (and with a margin) the two lie on the
// same side of the border (tests/test_corrected_quotient.py).  Scales from kCorrectedMin
// on keep the residual clear of underflow.  Worked on -1 / s, so that the order of
// the terms keeps the sign of a zero; the codes' sign bits are turned at the end.
constexpr float kCorrectedMin = 0x1p-90f;
struct Corrected {
    float2 nr, s;
};
FG8_DEV Corrected make_corrected(float s) {
    const float nr = -__frcp_rn(s);
    return {make_float2(nr, nr), make_float2(s, s)};
}
// -x / s
FG8_DEV float2 negated_quotient(float2 x, const Corrected& q) {
    const float2 nz = __fmul2_rn(x, q.nr);
    return __ffma2_rn(__ffma2_rn(nz, q.s, x), q.nr, nz);
}
// codes of eight values
FG8_DEV uint2 quant_corrected(float2 x0, float2 x1, float2 x2, float2 x3, const Corrected& q) {
    const float2 z0 = negated_quotient(x0, q), z1 = negated_quotient(x1, q);
    const float2 z2 = negated_quotient(x2, q), z3 = negated_quotient(x3, q);
    return make_uint2(__byte_perm(cvt_e4m3x2(z0.x, z0.y), cvt_e4m3x2(z1.x, z1.y), 0x5410) ^ 0x80808080u,
                      __byte_perm(cvt_e4m3x2(z2.x, z2.y), cvt_e4m3x2(z3.x, z3.y), 0x5410) ^ 0x80808080u);
}

// One 128-row tile of an expert in the padded token axis (tile number `tile`:
// padded columns from 128 * tile).
struct RowTile {
    int row0;   // first logical row
    int n_in;   // rows of the expert in it (<= 128; 0 if the offsets are not of this buffer)
    int tile;
};

// s_pref: exclusive prefix of tiles per expert (s_pref[E] = all tiles);
// offsets as the caller gave them; R rows exist.
FG8_DEV RowTile find_tile(int tile, const int32_t* s_pref, const int32_t* offsets, int E, int R) {
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_pref[mid] <= tile) lo = mid; else hi = mid;
    }
    const int64_t r0 = (int64_t)offsets[lo] + 128 * (int64_t)(tile - s_pref[lo]);
    RowTile t;
    t.tile = tile;
    t.row0 = r0 < 0 || r0 >= R ? 0 : (int)r0;
    // rows that the buffers do not hold (offsets inconsistent with R) are not touched
    t.n_in = r0 < 0 || r0 >= R ? 0 : (int)min((int64_t)min(128, R - t.row0), offsets[lo + 1] - r0);
    return t;
}

// Tiles per expert -> s_pref (exclusive prefix, s_pref[E] = total), by all
// threads of the block; s_warp: 33 words.
FG8_DEV void tile_prefix(const int32_t* offsets, int E, int32_t* s_pref, int32_t* s_warp) {
    for (int e = threadIdx.x; e < E; e += blockDim.x)
        s_pref[e] = (max(0, offsets[e + 1] - offsets[e]) + 127) / 128;
    __syncthreads();
    block_exclusive_scan(s_pref, s_pref, E, s_warp);
}

}  // namespace fg8
