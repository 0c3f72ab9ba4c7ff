// What the few-row products need of their rows (dq_rows_forward): the B operand
// and the low-rank factor's intermediate U = xv L1, in one launch.
//
//   B operand, by blocks of 4096 channels of a row.
//     FP4 form   eight digits a value (dq_rows_fp4.cu) and the first digit's unit
//     FP16 form  the value divided by a power of two E of its row, in FP16
//                (dq_rows.cu), with a scale per 64 channels as hi + lo halves
//     Each block finds the row's largest magnitude for itself: a second read of at
//     most 28 KB, from L2, costs less than a hand-off between blocks.
//   U, by clusters of eight CTAs for 16 rows and 32 ranks, an eighth of the
//     channels each (mma.sync; the work is small, its loads' latency is what
//     counts), joined in rank order through distributed shared memory and kept as
//     BF16 hi + lo, 2^-17 of the value: as it is for the FP4 form, whose product
//     has an accumulator of its own for it, divided by E S_W for the FP16 form,
//     whose accumulator has room for one.
#include "../../include/deltaquant.h"
#include "dq_common.h"
#include "dq_internal.h"
#include "dq_ptx.cuh"
#include "dq_rows.cuh"

namespace dq {

namespace {

constexpr int kThreads = 512, kCluster = 8, kBlockChannels = 8 * kThreads;

template <int kFmt, bool kDigitForm>
__device__ __forceinline__ void convert_block(const RowsParams& p, int m, int part) {
    __shared__ float sh[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, c = part * kBlockChannels + tid * 8;
    float am = 0.f;
    Raw8<kFmt> raw = {};
    if (c < p.Ci) raw = load_raw8<kFmt>(p, m, c);
    for (int i = tid * 8; i < p.Ci; i += kBlockChannels) am = max_nan(am, amax8<kFmt>(load_raw8<kFmt>(p, m, i)));
    griddep_launch();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
    if (lane == 0) sh[tid >> 5] = am;
    __syncthreads();
    am = sh[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; w++) am = max_nan(am, sh[w]);
    const bool finite = finite_row(am);
    const int k = row_unit<kFmt, kDigitForm>(am);
    if (part == 0 && tid == 0) {
        float E = k >= -126 ? pow2i(k) : __int_as_float(1 << (k + 149));
        if (kFmt == DQ_ROWS_E4M3) E *= p.x_scales[m];
        p.e[m] = finite ? E : __int_as_float(0x7FC00000);   // a NaN or an infinity: NaN all over the row
    }
    if (c >= p.Ci) return;
    float v[8];
    uint64_t v2[4];
    values8<kFmt>(raw, v);
    scaled_pairs(v, inv_scale(k), finite, v2);
    if (kDigitForm) {
        uint8_t* dst = (uint8_t*)p.xh + (size_t)m * kRowsDigits * (p.Ci / 2) + c / 2;
#pragma unroll
        for (int q = 0; q < kRowsDigits; q++) *reinterpret_cast<uint32_t*>(dst + (size_t)q * (p.Ci / 2)) = next_digits8(v2);
    } else {
        uint16_t* dst = p.xh + (size_t)m * (p.hilo ? 2 * p.Ci : p.Ci) + c;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            f2_unpack(v2[j], v[2 * j], v[2 * j + 1]);
            w[j] = f16x2_rn(v[2 * j], v[2 * j + 1]);
        }
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        if (kFmt == DQ_ROWS_E4M3_GROUP64) {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                float f0, f1;
                f16x2_values(w[j], f0, f1);
                w[j] = f16x2_rn(v[2 * j] - f0, v[2 * j + 1] - f1);
            }
            *reinterpret_cast<uint4*>(dst + p.Ci) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
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

template <int kFmt, bool kDigitForm>
__device__ __forceinline__ void lowrank_cluster(const RowsParams& p, int index) {
    __shared__ float wpart[8][16][32], part[16][32], wmax[8][16], cmax[16];
    __shared__ int rexp[16];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int crank = (int)cluster_ctarank(), rgroups = (p.rank + 31) / 32;
    const int m0 = index / rgroups * 16, nm = imin(16, p.rows - m0), j0 = index % rgroups * 32;
    const int nblk = p.Ci / 64, b0 = nblk * crank / kCluster, b1 = nblk * (crank + 1) / kCluster;
    // a warp takes 16 of the ranks and every eighth 64-channel block; lane t of a quad owns 16 channels of
    // a block (any assignment of channels to the MMA's k is right as long as both operands use it)
    const int jw = j0 + 16 * (warp & 1), ks = warp >> 1;
    const bool active = jw < p.rank;
    // L1's part for this CTA on its way before the product is let in: its streams of weights would come first
    for (int e = tid; e < imin(32, p.rank - j0) * (b1 - b0); e += kThreads) {
        const uint16_t* src = p.l1 + (long long)(j0 + e / (b1 - b0)) * p.Ci + (b0 + e % (b1 - b0)) * 64;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
    }
    griddep_launch();
    float acc[2][4] = {}, am[2] = {0.f, 0.f};
#pragma unroll 2
    for (int b = b0 + ks; b < b1; b += 8) {
        uint32_t xa[2][8];
        float sc[2];
        load_rows_16<kFmt>(p, m0, nm, b, g, t, xa, sc);
        if (!kDigitForm && kFmt != DQ_ROWS_E4M3) {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                float a = 0.f;
#pragma unroll
                for (int i = 0; i < 8; i++) a = max_nan(a, max_nan(fabsf(bf16_lo(xa[h][i])), fabsf(bf16_hi(xa[h][i]))));
                am[h] = max_nan(am[h], kFmt == DQ_ROWS_E4M3_GROUP64 ? fabsf(a * sc[h]) : a);
            }
        }
        if (active) {
#pragma unroll
            for (int n = 0; n < 2; n++) {
                const uint4* src = reinterpret_cast<const uint4*>(p.l1 + (long long)(jw + 8 * n + g) * p.Ci + b * 64 + t * 16);
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
    }
    // lane (g, t) holds the rows g, g + 8 and the ranks 8 n + 2 t, + 1 of its sixteen
#pragma unroll
    for (int n = 0; n < 2; n++) {
        float* w0 = &wpart[ks][g][16 * (warp & 1) + 8 * n + 2 * t];
        w0[0] = acc[n][0], w0[1] = acc[n][1];
        w0[8 * 32] = acc[n][2], w0[8 * 32 + 1] = acc[n][3];
    }
    if (!kDigitForm && kFmt != DQ_ROWS_E4M3) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) am[h] = max_nan(am[h], __shfl_xor_sync(0xffffffffu, am[h], o));
            if ((warp & 1) == 0 && t == 0) wmax[ks][g + 8 * h] = am[h];
        }
    }
    __syncthreads();
    {
        const int m = tid >> 5;
        float u = 0.f, a = 0.f;
#pragma unroll
        for (int k = 0; k < 8; k++) u += wpart[k][m][lane];
        part[m][lane] = u;
        if (!kDigitForm && kFmt != DQ_ROWS_E4M3 && tid < 16) {
#pragma unroll
            for (int k = 0; k < 8; k++) a = max_nan(a, wmax[k][tid]);
            cmax[tid] = a;
        }
    }
    cluster_sync();
    if (!kDigitForm) {
        if (tid < 16) {
            float a = 0.f;
            if (kFmt != DQ_ROWS_E4M3)
                for (int c = 0; c < kCluster; c++) a = max_nan(a, ld_dsmem_f32(mapa_shared(smem_u32(&cmax[tid]), c)));
            rexp[tid] = row_unit<kFmt, kDigitForm>(a);   // not finite: whatever it gives, the row's factor is NaN
        }
        __syncthreads();
    }
    // an eighth of the sums per CTA: two rows
    const int m = 2 * crank + ((tid >> 5) & 1), j = j0 + lane;
    uint16_t* dst = p.u + (long long)(m0 + m) * p.slab;
    if (tid < 64 && m < nm && j < p.rank) {
        const uint32_t at = smem_u32(&part[m][lane]);
        float u = 0.f;
#pragma unroll
        for (int c = 0; c < kCluster; c++) u += ld_dsmem_f32(mapa_shared(at, c));
        if (!kDigitForm) {
            const Scale2 s = inv_scale(rexp[m]);
            u = u / reinterpret_cast<const PackedHeader*>(p.packed_w)->S_W * s.a * s.b;
        } else if (kFmt == DQ_ROWS_E4M3) {
            u *= p.x_scales[m0 + m];
        }
        const uint16_t hi = f32_to_bf16_rn(u);
        dst[j] = hi;
        dst[p.rank + j] = f32_to_bf16_rn(u - bf16_lo(hi));
    } else if (tid >= 64 && tid < 128 && j0 == 0 && m < nm) {
        // zeros up to the slab's width (at most 32 columns)
        if (2 * p.rank + lane < p.slab) dst[2 * p.rank + lane] = 0;
    }
    cluster_sync();   // no CTA leaves while another still reads its sums
}

template <int kFmt, bool kDigitForm>
__global__ void __launch_bounds__(kThreads) k_rows_prepare(RowsParams p) {
    griddep_wait();     // the launch before this one may still read the workspace, or write X
    const int parts = (p.Ci + kBlockChannels - 1) / kBlockChannels, blocks = p.own_digits ? 0 : p.rows * parts;
    const int first = (blocks + kCluster - 1) / kCluster * kCluster, b = (int)blockIdx.x;
    if (b == first && threadIdx.x == 0) *p.status = header_ok(p) ? 0 : kStatusBadWeight;
    if (b >= first)
        lowrank_cluster<kFmt, kDigitForm>(p, (b - first) / kCluster);
    else if (b < blocks)
        convert_block<kFmt, kDigitForm>(p, b / parts, b % parts);
}

}  // namespace

cudaError_t launch_rows_prepare(const RowsParams& p, bool digit_form, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    const long long convert = p.own_digits ? 0 : cdiv((long long)p.rows * cdiv(p.Ci, kBlockChannels), kCluster);
    const long long low = cdiv(p.rows, 16) * cdiv(p.rank, 32);
    cfg.gridDim = dim3((unsigned)((convert + low) * kCluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    auto go = [&](auto kernel) {
        // the product's split of the SM between L1 and shared memory: a different one would keep its CTAs
        // off an SM until this kernel's have left
        const cudaError_t e = once_per_device((const void*)kernel, [&] {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        });
        return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kernel, p) : e;
    };
    if (digit_form) {
        if (p.x_format == DQ_ROWS_BF16) return go(k_rows_prepare<DQ_ROWS_BF16, true>);
        if (p.x_format == DQ_ROWS_E4M3) return go(k_rows_prepare<DQ_ROWS_E4M3, true>);
        return go(k_rows_prepare<DQ_ROWS_E4M3_GROUP64, true>);
    }
    if (p.x_format == DQ_ROWS_BF16) return go(k_rows_prepare<DQ_ROWS_BF16, false>);
    if (p.x_format == DQ_ROWS_E4M3) return go(k_rows_prepare<DQ_ROWS_E4M3, false>);
    return go(k_rows_prepare<DQ_ROWS_E4M3_GROUP64, false>);
}

}  // namespace dq
