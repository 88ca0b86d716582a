// mma_sync.cuh -- warp-level matrix helpers of the gated delta kernels: m16n8k16 bf16 products with
// fp32 accumulation, 8x8 matrix loads, 16-byte asynchronous copies, and the split of an fp32
// value into two or three bf16 terms.
//
// Fragments, with g = lane / 4 and c = lane % 4: an accumulator holds (row g, columns 2c, 2c+1) and
// (row g + 8, the same); operand A (16 x 16) is two such tiles side by side in bf16, and B (16 x 8)
// holds (rows 2c, 2c+1, column g) and (rows 2c + 8, 2c + 9).  An accumulator tile pair is therefore an
// A operand without any exchange between lanes, which is what keeps a memory's rows in registers.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace mc {
namespace mma {

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void stsm4t(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
                 : "memory");
}

__device__ __forceinline__ void stsm4(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
                 : "memory");
}

// The transpose of an 8 x 8 matrix of 16-bit values held as an accumulator tile in bf16 (row g, columns 2c, 2c + 1).
__device__ __forceinline__ uint32_t movm_t(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Copy 16 bytes to shared memory, or write zeros where `ok` is false (src is then not read).
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok)
{
    const int n = ok ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float low_f(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float high_f(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// x = hi + lo up to 2^-17 of x.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo)
{
    hi = pack2(x, y);
    lo = pack2(x - low_f(hi), y - high_f(hi));
}

// The same in three terms, up to 2^-25.
__device__ __forceinline__ void split3(float x, float y, uint32_t &hi, uint32_t &mid, uint32_t &lo)
{
    hi = pack2(x, y);
    split2(x - low_f(hi), y - high_f(hi), mid, lo);
}

// Byte offset of 16-byte piece c of row r in a tile of rows of ROW bytes (a multiple of 128): pieces are
// exchanged within their 128 bytes by the row, so that eight rows of a column touch every bank once.
template <int ROW>
__device__ __forceinline__ uint32_t tile_off(int r, int c)
{
    return (uint32_t)(r * ROW + ((c & ~7) << 4) + (((c ^ r) & 7) << 4));
}

}  // namespace mma
}  // namespace mc
