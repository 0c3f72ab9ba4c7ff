// Pieces shared by the two forms of the few-row product (dq_rows_fp4.cu, dq_rows.cu) and what prepares their
// rows (dq_rows_prep.cu).
#pragma once

#include <atomic>

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

// Two E4M3 codes -> FP16 pair (exact), the low byte's in the low half
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)codes));
    return h2;
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

// The next FP4 digit of each of eight values |v| <= 4 (as four fp32 pairs) as packed codes: the nearest
// integers, which the values then leave for the next digit, eight times finer.  Every step is exact.
__device__ __forceinline__ uint32_t next_digits8(uint64_t (&v)[4]) {
    const uint64_t magic = f2_pack(12582912.f, 12582912.f), eight = f2_pack(8.f, 8.f);   // 1.5 2^23
    float d[8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint64_t n = f2_sub(f2_add(v[i], magic), magic);
        v[i] = f2_mul(f2_sub(v[i], n), eight);
        f2_unpack(n, d[2 * i], d[2 * i + 1]);
    }
    return cvt_e2m1x8(d);
}

// Eight channels of a row as they lie in memory, and their values
template <int kFmt>
struct Raw8 {
    uint32_t w[kFmt == DQ_ROWS_BF16 ? 4 : 2];
    float s;   // the scale of their 64 channels
};

// Channels c to c + 7 of row m
template <int kFmt>
__device__ __forceinline__ Raw8<kFmt> load_raw8(const RowsParams& p, int m, int c) {
    Raw8<kFmt> r;
    const long long off = (long long)m * p.x_stride + c;
    if (kFmt == DQ_ROWS_BF16) {
        const uint4 a = *reinterpret_cast<const uint4*>((const uint16_t*)p.x + off);
        r.w[0] = a.x, r.w[1] = a.y, r.w[kFmt == DQ_ROWS_BF16 ? 2 : 0] = a.z, r.w[kFmt == DQ_ROWS_BF16 ? 3 : 0] = a.w;
    } else {
        const uint2 a = *reinterpret_cast<const uint2*>((const uint8_t*)p.x + off);
        r.w[0] = a.x, r.w[1] = a.y;
    }
    r.s = kFmt == DQ_ROWS_E4M3_GROUP64 ? p.x_scales[(long long)m * (p.Ci / 64) + c / 64] : 1.f;
    return r;
}

template <int kFmt>
__device__ __forceinline__ void values8(const Raw8<kFmt>& r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (kFmt == DQ_ROWS_BF16) {
            v[2 * i] = bf16_lo(r.w[i % (kFmt == DQ_ROWS_BF16 ? 4 : 2)]), v[2 * i + 1] = bf16_hi(r.w[i % (kFmt == DQ_ROWS_BF16 ? 4 : 2)]);
        } else {
            f16x2_values(e4m3x2_to_f16x2(r.w[i / 2] >> (16 * (i & 1))), v[2 * i], v[2 * i + 1]);
            if (kFmt == DQ_ROWS_E4M3_GROUP64) v[2 * i] *= r.s, v[2 * i + 1] *= r.s;
        }
    }
}

template <int kFmt>
__device__ __forceinline__ float amax8(const Raw8<kFmt>& r) {
    float v[8];
    values8<kFmt>(r, v);
    float a = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < 8; i++) a = max_nan(a, fabsf(v[i]));
    return a;
}

// Exponent k of a row's power of two E = 2^k from its largest magnitude: the first digit's unit (values
// below 4 units), or what moves the row to at most 2^15; subnormals count as 2^-126.  E4M3 codes need none in
// the FP16 form.
template <int kFmt, bool kDigitForm>
__device__ __forceinline__ int row_unit(float am) {
    if (!kDigitForm && kFmt == DQ_ROWS_E4M3) return 0;
    const int e = (int)((__float_as_uint(am) >> 23) & 255);
    return (e ? e - 127 : -126) - (kDigitForm ? 1 : 14);
}

__device__ __forceinline__ bool finite_row(float am) { return am < __int_as_float(0x7F800000); }

// v 2^-k in two exact steps (k in [-140, 126])
struct Scale2 {
    float a, b;
};
__device__ __forceinline__ Scale2 inv_scale(int k) {
    const int h = (-k) / 2;
    return Scale2{pow2i(h), pow2i(-k - h)};
}

// v 2^-k for eight values (zeros for a row that is not finite: its factor is NaN)
__device__ __forceinline__ void scaled_pairs(const float (&v)[8], Scale2 s, bool finite, uint64_t (&o)[4]) {
    const uint64_t a = f2_pack(s.a, s.a), b = f2_pack(s.b, s.b);
#pragma unroll
    for (int i = 0; i < 4; i++) o[i] = finite ? f2_mul(f2_mul(f2_pack(v[2 * i], v[2 * i + 1]), a), b) : 0ull;
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

// Runs `set` (a kernel's attributes) on the first call for that kernel on the current device.  Concurrent
// first calls may both run it; they set the same values.
template <typename Set>
inline cudaError_t once_per_device(const void* kernel, Set set) {
    constexpr int kKernels = 32, kDevices = 64;
    static std::atomic<const void*> names[kKernels];
    static std::atomic<uint64_t> done[kKernels];   // a bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int i = 0;
    for (; i < kKernels; i++) {
        const void* at = names[i].load(std::memory_order_acquire);
        if (at == nullptr && !names[i].compare_exchange_strong(at, kernel)) at = names[i].load(std::memory_order_acquire);
        if (at == nullptr || at == kernel) break;
    }
    if (i == kKernels || dev >= kDevices) return set();
    if (done[i].load(std::memory_order_acquire) >> dev & 1) return cudaSuccess;
    if ((e = set()) == cudaSuccess) done[i].fetch_or(1ull << dev, std::memory_order_release);
    return e;
}

}  // namespace dq
