// quant_tile.cuh -- the 128 x 128 bf16 tile in shared memory that the quantizer kernels work
// on: two boxes of 64 columns (128 bytes) a row, 16-byte chunks XOR-swizzled by row, its
// shared-memory reads, and the E2M1 codes of a column pair.
#pragma once

#include <cstdint>

namespace mxfp4 {

constexpr int kQT = 128;                       // tile edge (rows and columns)
constexpr int kQTileBytes = kQT * kQT * 2;
constexpr int kQBoxBytes = kQT * 128;          // 128 rows x 64 bf16 columns

// Byte offset of (row r, 16-byte chunk j of the 128-byte box row) under the 128-byte
// swizzle: chunk j of row r is stored at chunk j ^ (r % 8).
__device__ __forceinline__ uint32_t swz(int r, int j) { return r * 128 + ((j ^ (r & 7)) << 4); }

// Eight words = rows 2j, 2j+1 (j = 0..3) of a column pair (column c0 in the low halves,
// c1 in the high halves), times the pair's scales `s2` = {s(c0), s(c1)}: four bytes of
// codes for c0 (*q0) and for c1 (*q1), row 2j in the low nibble of byte j.
__device__ __forceinline__ void encode_cols8(const uint32_t* w, uint64_t s2, uint32_t* q0,
                                             uint32_t* q1) {
    asm("{\n\t"
        ".reg .b32 l<8>, h<8>;\n\t"
        ".reg .b64 x<8>;\n\t"
        ".reg .f32 a<8>, b<8>;\n\t"
        ".reg .b8 c<4>, d<4>;\n\t"
        "shl.b32 l0, %2, 16;\n\tand.b32 h0, %2, 0xFFFF0000;\n\t"
        "shl.b32 l1, %3, 16;\n\tand.b32 h1, %3, 0xFFFF0000;\n\t"
        "shl.b32 l2, %4, 16;\n\tand.b32 h2, %4, 0xFFFF0000;\n\t"
        "shl.b32 l3, %5, 16;\n\tand.b32 h3, %5, 0xFFFF0000;\n\t"
        "shl.b32 l4, %6, 16;\n\tand.b32 h4, %6, 0xFFFF0000;\n\t"
        "shl.b32 l5, %7, 16;\n\tand.b32 h5, %7, 0xFFFF0000;\n\t"
        "shl.b32 l6, %8, 16;\n\tand.b32 h6, %8, 0xFFFF0000;\n\t"
        "shl.b32 l7, %9, 16;\n\tand.b32 h7, %9, 0xFFFF0000;\n\t"
        "mov.b64 x0, {l0, h0};\n\tmov.b64 x1, {l1, h1};\n\t"
        "mov.b64 x2, {l2, h2};\n\tmov.b64 x3, {l3, h3};\n\t"
        "mov.b64 x4, {l4, h4};\n\tmov.b64 x5, {l5, h5};\n\t"
        "mov.b64 x6, {l6, h6};\n\tmov.b64 x7, {l7, h7};\n\t"
        "mul.rn.f32x2 x0, x0, %10;\n\tmul.rn.f32x2 x1, x1, %10;\n\t"
        "mul.rn.f32x2 x2, x2, %10;\n\tmul.rn.f32x2 x3, x3, %10;\n\t"
        "mul.rn.f32x2 x4, x4, %10;\n\tmul.rn.f32x2 x5, x5, %10;\n\t"
        "mul.rn.f32x2 x6, x6, %10;\n\tmul.rn.f32x2 x7, x7, %10;\n\t"
        "mov.b64 {a0, b0}, x0;\n\tmov.b64 {a1, b1}, x1;\n\t"
        "mov.b64 {a2, b2}, x2;\n\tmov.b64 {a3, b3}, x3;\n\t"
        "mov.b64 {a4, b4}, x4;\n\tmov.b64 {a5, b5}, x5;\n\t"
        "mov.b64 {a6, b6}, x6;\n\tmov.b64 {a7, b7}, x7;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c0, a1, a0;\n\tcvt.rn.satfinite.e2m1x2.f32 d0, b1, b0;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c1, a3, a2;\n\tcvt.rn.satfinite.e2m1x2.f32 d1, b3, b2;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c2, a5, a4;\n\tcvt.rn.satfinite.e2m1x2.f32 d2, b5, b4;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c3, a7, a6;\n\tcvt.rn.satfinite.e2m1x2.f32 d3, b7, b6;\n\t"
        "mov.b32 %0, {c0, c1, c2, c3};\n\t"
        "mov.b32 %1, {d0, d1, d2, d3};\n\t}"
        : "=r"(*q0), "=r"(*q1)
        : "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]),
          "l"(s2));
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a));
    return v;
}

}  // namespace mxfp4
