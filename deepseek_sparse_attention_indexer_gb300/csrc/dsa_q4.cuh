// dsa_q4.cuh -- the 4-bit cache row and its expansion, shared by the kernels
// that write, read and attend over it.
//
// A row is 416 bytes: 512 codes of four bits | 32 block bytes | 64 bf16 rope dims.  A code is a sign and one of the
// magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6; block byte 3 a + m scales the codes of 16 dims by (1 + m / 4) 2^(a - 6), m < 3,
// a < 12 (36 and above: zeros).  The three fractions are those whose product with every magnitude has four significant
// bits, and the twelve powers those whose products end within e4m3's range: every value of a row is an e4m3 number times
// the row's scale.  A word of eight dims has the magnitude of dim i in bits 4 i .. 4 i + 2, as a byte selector takes
// them, and the signs of dims i and 4 + i in bits 8 i + 7 and 8 i + 3, where a shift by 0 or 4 puts them on e4m3 bytes'.
#pragma once
#include "dsa_q8.cuh"

namespace dsa {

constexpr int kQ4Row = DSA_Q4_ROW_BYTES;
constexpr int kQ4Codes = DSA_V_DIM / 2;            // bytes of the codes; the block bytes follow
constexpr int kQ4Block = 16;                       // dims of a block
constexpr int kQ4Blocks = DSA_V_DIM / kQ4Block;    // 32
constexpr int kQ4Rope = kQ4Codes + kQ4Blocks;      // offset of the rope dims
constexpr int kQ4Scales = 36;                      // block bytes in use
static_assert(kQ4Row == kQ4Rope + 2 * kQ8Rope && kQ4Row % 32 == 0 && kQ4Rope % 32 == 0, "a 4-bit cache row");

constexpr uint32_t kQ4Magnitudes = 0x77777777u;    // of a word of eight codes

__device__ __forceinline__ float q4_block_scale(uint32_t byte) {   // of a block byte below 36
    return (1.f + 0.25f * (float)(byte % 3)) * exp2_int((int)(byte / 3) - 6);
}
// The eight magnitudes times x as e4m3 bytes (exact for a block's scale)
__device__ __forceinline__ uint2 q4_table(float x) {
    return make_uint2(pack_e4m3x4(0.f, 0.5f * x, x, 1.5f * x), pack_e4m3x4(2.f * x, 3.f * x, 4.f * x, 6.f * x));
}
// The bytes of (x, y) that the low four nibbles of sel name, each below 8 (an instruction; the intrinsic masks first)
__device__ __forceinline__ uint32_t select_bytes(uint32_t x, uint32_t y, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(sel));
    return r;
}
// Eight codes as e4m3 bytes, by the table of their block
__device__ __forceinline__ uint2 q4_expand(uint32_t w, uint2 table) {
    const uint32_t sel = w & kQ4Magnitudes;
    return make_uint2(select_bytes(table.x, table.y, sel) | (w & 0x80808080u),
                      select_bytes(table.x, table.y, sel >> 16) | ((w << 4) & 0x80808080u));
}

}  // namespace dsa
