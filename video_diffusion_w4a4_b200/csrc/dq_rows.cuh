// Pieces shared by the two forms of the few-row product (dq_rows.cu, dq_rows_direct.cu).
#pragma once

#include "../../include/deltaquant.h"
#include "dq_internal.h"
#include "dq_ptx.cuh"

namespace dq {

constexpr uint32_t kRowsCodeBytes = 128 * 128;   // codes of 128 output channels x 256 input channels
constexpr uint32_t kRowsScaleBytes = 4 * 512;    // their group scales
constexpr int kRowsStages = 16;                  // stages of an operand ring at most

__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// D(16 x 8) += A(16 x 16) B(16 x 8), BF16 operands, fp32 sums
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two E4M3 codes -> FP16 pair (exact), the low byte's in the low half
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)codes));
    return h2;
}

// Eight E2M1 codes (value 2i in the low nibble of byte i) times the FP16 pair s -> four FP16 pairs
__device__ __forceinline__ void decode8(uint32_t w, uint32_t s, uint32_t* out) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        ".reg .b32 t0, t1, t2, t3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 t0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 t1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 t2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 t3, b3;\n\t"
        "mul.rn.f16x2 %0, t0, %5;\n\t"
        "mul.rn.f16x2 %1, t1, %5;\n\t"
        "mul.rn.f16x2 %2, t2, %5;\n\t"
        "mul.rn.f16x2 %3, t3, %5;\n\t}"
        : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
        : "r"(w), "r"(s));
}

__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ bool header_ok(const RowsParams& p) {
    const PackedHeader* h = reinterpret_cast<const PackedHeader*>(p.packed_w);
    return h->magic == DQ_PACK_MAGIC && h->version == DQ_PACK_FORMAT_VERSION && h->Ci == p.Ci && h->Co == p.Co &&
           h->rank == p.rank && h->slab == p.slab;
}

__device__ __forceinline__ void f16x2_values(uint32_t h2, float& lo, float& hi) {
    __half2_raw r;
    r.x = (uint16_t)(h2 & 0xFFFFu), r.y = (uint16_t)(h2 >> 16);
    const float2 f = __half22float2(__half2(r));
    lo = f.x, hi = f.y;
}

// The power of two that moves a BF16 row (largest magnitude am > 0, finite) into FP16's range: am / 2^k
// in [2^14, 2^15); a subnormal am is taken as 2^-126.
__device__ __forceinline__ int row_exponent(float am) {
    const int e = (int)((__float_as_uint(am) >> 23) & 255);
    return (e ? e - 127 : -126) - 14;
}

// Channels 64 b + 16 t to + 15 of the rows m0 + g and m0 + g + 8 as BF16 pairs (zeros from row nm on), and
// their scales where the format has one per 64 channels.
template <int kFmt>
__device__ __forceinline__ void load_rows_16(const RowsParams& p, int m0, int nm, int b, int g, int t, uint32_t (&xa)[2][8],
                                             float (&sc)[2]) {
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int m = g + 8 * h;
#pragma unroll
        for (int i = 0; i < 8; i++) xa[h][i] = 0;
        sc[h] = 0.f;
        if (m >= nm) continue;
        const long long off = (long long)(m0 + m) * p.x_stride + b * 64 + t * 16;
        if (kFmt == DQ_ROWS_BF16) {
            const uint4* src = reinterpret_cast<const uint4*>((const uint16_t*)p.x + off);
            const uint4 u = src[0], v = src[1];
            xa[h][0] = u.x, xa[h][1] = u.y, xa[h][2] = u.z, xa[h][3] = u.w;
            xa[h][4] = v.x, xa[h][5] = v.y, xa[h][6] = v.z, xa[h][7] = v.w;
        } else {
            const uint4 u = *reinterpret_cast<const uint4*>((const uint8_t*)p.x + off);
            const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 8; i++) xa[h][i] = e4m3x2_to_bf16x2(q[i / 2] >> (16 * (i & 1)));
        }
        if (kFmt == DQ_ROWS_E4M3_GROUP64) sc[h] = p.x_scales[(long long)(m0 + m) * (p.Ci / 64) + b];
    }
}

// acc[n] += X L1 over the 64 channels of block b, ranks 8 n to 8 n + 7 (any assignment of channels to the MMA's
// k is right as long as both operands use it)
template <int kNT, int kFmt>
__device__ __forceinline__ void lowrank_block(const RowsParams& p, int b, int g, int t, const uint32_t (&xa)[2][8],
                                              const float (&sc)[2], float (&acc)[kNT][4]) {
#pragma unroll
    for (int n = 0; n < kNT; n++) {
        if (8 * n >= p.rank) break;
        const uint4* src = reinterpret_cast<const uint4*>(p.l1 + (long long)(8 * n + g) * p.Ci + b * 64 + t * 16);
        const uint4 u = src[0], v = src[1];
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma_16816(d, xa[0][0], xa[1][0], xa[0][1], xa[1][1], u.x, u.y);
        mma_16816(d, xa[0][2], xa[1][2], xa[0][3], xa[1][3], u.z, u.w);
        mma_16816(d, xa[0][4], xa[1][4], xa[0][5], xa[1][5], v.x, v.y);
        mma_16816(d, xa[0][6], xa[1][6], xa[0][7], xa[1][7], v.z, v.w);
        const float s0 = kFmt == DQ_ROWS_E4M3_GROUP64 ? sc[0] : 1.f, s1 = kFmt == DQ_ROWS_E4M3_GROUP64 ? sc[1] : 1.f;
        acc[n][0] = fmaf(d[0], s0, acc[n][0]);
        acc[n][1] = fmaf(d[1], s0, acc[n][1]);
        acc[n][2] = fmaf(d[2], s1, acc[n][2]);
        acc[n][3] = fmaf(d[3], s1, acc[n][3]);
    }
}

// Lane (g, t) holds U of rows g, g + 8 and ranks 8 n + 2 t, + 1: into a 16 x rank array
template <int kNT>
__device__ __forceinline__ void store_lowrank(float* dst, int rank, int g, int t, const float (&acc)[kNT][4]) {
#pragma unroll
    for (int n = 0; n < kNT; n++) {
        if (8 * n >= rank) break;
        float* w0 = dst + g * rank + 8 * n + 2 * t;
        w0[0] = acc[n][0], w0[1] = acc[n][1];
        w0[8 * rank] = acc[n][2], w0[8 * rank + 1] = acc[n][3];
    }
}

// A place in a ring and the parity of its use, stepped without a division (a division by a runtime
// ring size costs more than a chunk's MMAs)
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int size) {
        if (++slot == size) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// One lane's wait for the whole warp
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                          uint64_t budget_ns) {
    bool ok = true;
    if ((threadIdx.x & 31) == 0) ok = mbar_wait_spin(bar, parity, abort_flag, status, budget_ns);
    return __shfl_sync(0xffffffffu, ok, 0);
}

// One lane of a converged warp, the same every time
__device__ __forceinline__ bool elect_one() {
    uint32_t pred;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(pred));
    return pred != 0;
}

__device__ __forceinline__ float ld_dsmem_f32(uint32_t cluster_addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_dsmem_f32(uint32_t cluster_addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}

}  // namespace dq
