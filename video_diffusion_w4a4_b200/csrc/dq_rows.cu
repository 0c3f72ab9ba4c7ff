// The product of few rows with a packed 4-bit weight (dq_rows_forward):
//   Y[m] = act( S_W sum_c xv[m][c] (q s_b)[o][c] + (xv[m] L1) L2 + b )
#include "../../include/deltaquant.h"
#include "dq_common.h"
#include "dq_internal.h"
#include "dq_ptx.cuh"

namespace dq {

namespace {

__device__ __forceinline__ bool header_ok(const RowsParams& p) {
    const PackedHeader* h = reinterpret_cast<const PackedHeader*>(p.packed_w);
    return h->magic == DQ_PACK_MAGIC && h->version == DQ_PACK_FORMAT_VERSION && h->Ci == p.Ci && h->Co == p.Co &&
           h->rank == p.rank && h->slab == p.slab;
}

__device__ __forceinline__ float x_value(const RowsParams& p, int m, int c) {
    if (p.x_format == DQ_ROWS_BF16) return bf16_lo(((const uint16_t*)p.x)[(long long)m * p.x_stride + c]);
    const float v = e4m3_to_f32(((const uint8_t*)p.x)[(long long)m * p.x_stride + c]);
    return v * (p.x_format == DQ_ROWS_E4M3 ? p.x_scales[m] : p.x_scales[(long long)m * (p.Ci / 64) + c / 64]);
}

__device__ __forceinline__ float warp_sum(float v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// U[m][j] = sum_c xv[m][c] L1[j][c]: one warp each
__global__ void __launch_bounds__(256) k_rows_u(RowsParams p) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = header_ok(p) ? 0 : kStatusBadWeight;
    const int m = blockIdx.x, j = blockIdx.y * 8 + (threadIdx.x >> 5);
    float u = 0.f;
    for (int c = threadIdx.x & 31; c < p.Ci; c += 32) u = fmaf(x_value(p, m, c), bf16_lo(p.l1[(long long)j * p.Ci + c]), u);
    u = warp_sum(u);
    if ((threadIdx.x & 31) == 0) p.u[(long long)m * p.rank + j] = u;
}

// One output value per warp
__global__ void __launch_bounds__(256) k_rows_simple(RowsParams p) {
    if (!header_ok(p)) return;
    const int o = blockIdx.x * 8 + (threadIdx.x >> 5), m = blockIdx.y, lane = threadIdx.x & 31;
    const uint8_t* codes = p.packed_w + p.off_codes + (long long)o * (p.Ci / 2);
    float acc = 0.f;
    for (int b = lane; b < p.Ci / 16; b += 32) {
        const float s = e4m3_to_f32(p.packed_w[p.off_scales + sfb_offset(o, b, p.Ci)]);
        float part = 0.f;
        for (int i = 0; i < 16; i++) {
            const int q = (codes[b * 8 + i / 2] >> (4 * (i & 1))) & 15, e = (q >> 1) & 3;
            const float mag = e ? (1.f + 0.5f * (q & 1)) * (float)(1 << e) * 0.5f : 0.5f * (q & 1);
            part = fmaf(x_value(p, m, b * 16 + i), q & 8 ? -mag : mag, part);
        }
        acc = fmaf(part, s, acc);
    }
    float low = 0.f;
    for (int j = lane; j < p.rank; j += 32) low = fmaf(p.u[(long long)m * p.rank + j], bf16_lo(p.l2[(long long)o * p.slab + j]), low);
    acc = warp_sum(acc);
    low = warp_sum(low);
    if (lane) return;
    const PackedHeader* h = reinterpret_cast<const PackedHeader*>(p.packed_w);
    float y = acc * h->S_W + low;
    if (h->flags & kPackedHasBias) y += *(const float*)(p.packed_w + p.off_bias + 4ll * o);
    if (p.gelu) {
        float g, unused;
        f2_unpack(gelu_erf2(f2_pack(y, 0.f)), g, unused);
        y = g;
    }
    p.y[(long long)m * p.y_stride + o] = f32_to_bf16_rn(y);
}

}  // namespace

cudaError_t launch_rows(const RowsParams& p, cudaStream_t st) {
    k_rows_u<<<dim3(p.rows, p.rank / 8), 256, 0, st>>>(p);
    k_rows_simple<<<dim3(p.Co / 8, p.rows), 256, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace dq
