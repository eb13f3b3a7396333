// attn_frag.cuh -- what the mma.sync attention kernels share (the contiguous
// cache's split kernel and the paged one): programmatic launches, ldmatrix and
// mma.sync fragments, and codes as exact fp16 operands.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace srftkv {

// Programmatic dependent launch.  A kernel launched with programmatic stream
// serialisation may start while the kernel before it in the stream still runs;
// griddep_wait blocks until that kernel has completed and its memory writes are
// visible (a no-op for a kernel launched the ordinary way).  griddep_launch_dependents
// lets the next such kernel start launching once every CTA of this one has
// called it or exited.
__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void griddep_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// two matrices (the addresses of lanes 0-15)
__device__ __forceinline__ void ldsm_x2(uint32_t addr, uint32_t (&r)[2]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_x2_t(uint32_t addr, uint32_t (&r)[2]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// D = A . B + D, m16n8k16, fp16 inputs, fp32 accumulators
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D = A . B + (c0, c1, c0, c1): the accumulator starts from per-column values
__device__ __forceinline__ void mma16816_c(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                           uint32_t b0, uint32_t b1, float c0, float c1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %10, %11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
// (a, b) ~= hi + lo with both halves fp16: the MMA then sees a and b to about
// 22 bits instead of 11 (codes are exact in fp16, so this is the only rounding
// of the contraction inputs).
// The residuals a - hi.x and b - hi.y are exact in fp32 (hi is a rounding of
// them to 11 bits); each is one mixed-precision FMA, hi.x * -1 + a, with the
// fp16 half taken straight from the packed register instead of a widening
// convert and a subtraction.
__device__ __forceinline__ void split_h2(float a, float b, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(a, b);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    float ra, rb;
    asm("{\n\t.reg .f16 hx, hy, m1;\n\t"
        "mov.b32 {hx, hy}, %2;\n\t"
        "mov.b16 m1, 0xBC00;\n\t"
        "fma.rn.f32.f16 %0, hx, m1, %3;\n\t"
        "fma.rn.f32.f16 %1, hy, m1, %4;\n\t}"
        : "=f"(ra), "=f"(rb)
        : "r"(hi), "f"(a), "f"(b));
    const __half2 l = __floats2half2_rn(ra, rb);
    lo = *reinterpret_cast<const uint32_t*>(&l);
}
// Packed fp32 (one instruction for two lanes of work; IEEE rounding per lane).
__device__ __forceinline__ float2 mul2(float a0, float a1, float b0, float b1) {
    return __fmul2_rn(make_float2(a0, a1), make_float2(b0, b1));
}
__device__ __forceinline__ float2 fma2(float a0, float a1, float b0, float b1, float2 c) {
    return __ffma2_rn(make_float2(a0, a1), make_float2(b0, b1), c);
}

// Codes -> fp16 pairs in one logic op.  Bits 0xF/0xF0000 (0xF0/0xF00000)
// hold two two's-complement nibbles; XOR with 8 makes them offset binary, and
// with a zero exponent field the fp16 bit pattern is the subnormal
// (q + 8) * 2^-24 (or (q + 8) * 2^-20 for the high nibbles), exactly.  Bytes
// give (q + 128) * 2^-24.  The offset is removed after the contraction from the
// column sums of the other operand (offset * sum of B), which is small enough
// next to the signal that nothing is lost to cancellation; the unit 2^-24 is
// folded into the score and output scaling.
constexpr float kSub = 16777216.f;  // 2^24
// The XOR to offset binary is taken once per loaded word (ob4 / ob8: every
// nibble or byte at once, and it commutes with the >> 8 of the second pair),
// so each extraction is a single AND: (w & m) ^ (0x8.. & m) as one logic op
// would need two immediate operands, which one LOP3 cannot take.
__device__ __forceinline__ uint32_t ob4(uint32_t w) { return w ^ 0x88888888u; }  // int4 nibbles -> offset binary
__device__ __forceinline__ uint32_t ob8(uint32_t w) { return w ^ 0x80808080u; }  // int8 bytes -> offset binary
__device__ __forceinline__ uint32_t u4_lo(uint32_t wx) { return wx & 0x000F000Fu; }  // nibbles 0, 16 of ob4(w)
__device__ __forceinline__ uint32_t u4_hi(uint32_t wx) { return wx & 0x00F000F0u; }  // nibbles 4, 20 of ob4(w)
__device__ __forceinline__ uint32_t u8_lo(uint32_t wx) { return wx & 0x00FF00FFu; }  // bytes 0, 2 of ob8(w)
__device__ __forceinline__ float h2_sum(uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return f.x + f.y;
}

__device__ __forceinline__ float ex2(float x) {  // 2^x; ex2.approx has a relative error of about 2^-22
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace srftkv
