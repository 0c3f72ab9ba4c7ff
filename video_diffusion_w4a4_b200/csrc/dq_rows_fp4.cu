// The product of few rows with a packed 4-bit weight on the block-scaled FP4
// tensor cores (dq_rows_forward; dq_rows.cu has the form for more rows).
//
// Few rows leave the weight's bytes as the bound, and decoding codes costs more
// time than reading them.  Here they are not decoded: codes and group scales are
// the A operand of kind::mxf4nvf4 as they lie in the packed weight, and the rows
// of X are written exactly enough in the same format.  A group of 16 values with
// largest magnitude in [2^e, 2^(e+1)) is a sum of kDigits = 6 FP4 digits,
//   x = 2^(e-1) sum_p 8^-p d_p + r,   d_p in {-4, ..., 4},  |r| <= 2^(e-17),
// d_p the nearest integer to what the digits before it leave.  A BF16 value at
// least 2^-9 of its group's largest is exact, a smaller one off by at most 2^-17
// of the largest; so are E4M3 codes (those are exact down to 2^-13), and code *
// scale with a scale per 64 channels.  All digits of a group carry the scale
// 2^(e-1) / E as E4M3 (2^-9 to 2^8, with E the row's power of two; a group below
// 2^-17 of the row's largest is held relative to that), each digit is a column of
// the MMA, and the epilogue sums a row's columns with their weights 8^-p in fp32.
//
//   k_rows_digits   per row: digits, scales, E; beside it U = xv L1 in up to 16
//                   partial sums over the channels (mma.sync)
//   k_rows_fp4      128 output channels (the MMA's M) times up to 40 rows (240
//                   columns) per CTA.  One warp keeps codes and scales in flight,
//                   one the digits, one lane issues scale copies and MMAs; when
//                   the tiles alone do not fill the GPU a cluster splits the
//                   channels and sums its parts in rank order through distributed
//                   shared memory.  Its loads of the weight do not wait for
//                   k_rows_digits (programmatic launch).
#include "../../include/deltaquant.h"
#include "dq_common.h"
#include "dq_internal.h"
#include "dq_ptx.cuh"
#include "dq_rows.cuh"

namespace dq {

namespace {

constexpr int kDigits = kRowsDigits;

// ------------------------------------------------------------------ rows -> digits, and U

constexpr int kPrepThreads = 256;

// The values of 16 consecutive channels (group grp) of row m
template <int kFmt>
__device__ __forceinline__ void load_values16(const RowsParams& p, int m, int grp, float (&v)[16]) {
    const long long off = (long long)m * p.x_stride + grp * 16;
    if (kFmt == DQ_ROWS_BF16) {
        const uint4* src = reinterpret_cast<const uint4*>((const uint16_t*)p.x + off);
        const uint4 a = src[0], b = src[1];
        const uint32_t r[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; i++) v[2 * i] = bf16_lo(r[i]), v[2 * i + 1] = bf16_hi(r[i]);
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>((const uint8_t*)p.x + off);
        const uint32_t r[4] = {a.x, a.y, a.z, a.w};
        const float s = kFmt == DQ_ROWS_E4M3_GROUP64 ? p.x_scales[(long long)m * (p.Ci / 64) + grp / 4] : 1.f;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            f16x2_values(e4m3x2_to_f16x2(r[i / 2] >> (16 * (i & 1))), v[2 * i], v[2 * i + 1]);
            if (kFmt == DQ_ROWS_E4M3_GROUP64) v[2 * i] *= s, v[2 * i + 1] *= s;
        }
    }
}

__device__ __forceinline__ float amax16(const float (&v)[16]) {
    float a = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < 16; i++) a = max_nan(a, fabsf(v[i]));
    return a;
}

// floor(log2 a), -126 for subnormals and zero
__device__ __forceinline__ int exponent_of(float a) {
    const int e = (int)((__float_as_uint(a) >> 23) & 255);
    return e ? e - 127 : -126;
}

template <int kFmt>
__device__ __forceinline__ void digits_of_row(const RowsParams& p, int m) {
    __shared__ float sh[kPrepThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, groups = p.Ci / 16;
    float v[16], am = 0.f;
    for (int g = tid; g < groups; g += kPrepThreads) {
        load_values16<kFmt>(p, m, g, v);
        am = max_nan(am, amax16(v));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
    if (lane == 0) sh[tid >> 5] = am;
    __syncthreads();
    am = sh[0];
#pragma unroll
    for (int w = 1; w < kPrepThreads / 32; w++) am = max_nan(am, sh[w]);
    const bool finite = am < __int_as_float(0x7F800000);
    const int K = exponent_of(am) - 9;              // E = 2^K; the largest group's scale is 2^8
    if (tid == 0) {
        float E = K >= -126 ? pow2i(K) : __int_as_float(1 << (K + 149));
        if (kFmt == DQ_ROWS_E4M3) E *= p.x_scales[m];
        p.e[m] = finite ? E : __int_as_float(0x7FC00000);   // a NaN or an infinity: NaN all over the row
    }
    const int pass = m / p.n_rows, n0 = (m - pass * p.n_rows) * kDigits;   // the row's first column of its pass
    uint8_t* codes = (uint8_t*)p.xh + (size_t)m * kDigits * (p.Ci / 2);
    uint8_t* scales = p.x_sf + (size_t)pass * (p.Ci / 64) * p.sf_groups * 512;
    // groups is a multiple of 16, so the four groups of a 64-channel block are in four lanes of one warp
    for (int g = tid; g < groups; g += kPrepThreads) {
        load_values16<kFmt>(p, m, g, v);
        const float a = amax16(v);
        int j = exponent_of(a) - 1 - K;             // scale 2^j, j <= 8
        j = j < -9 ? -9 : j;
        const uint32_t code = j >= -6 ? (uint32_t)(j + 7) << 3 : 4u >> (-7 - j);
        const int k = -(K + j), h = k / 2;          // |value 2^k| < 4; k in [-126, 136]: two exact steps
        const float f0 = pow2i(h), f1 = pow2i(k - h);
#pragma unroll
        for (int i = 0; i < 16; i++) v[i] = finite ? v[i] * f0 * f1 : 0.f;
        uint8_t* dst = codes + g * 8;
#pragma unroll
        for (int q = 0; q < kDigits; q++) {
            float d[16];
#pragma unroll
            for (int i = 0; i < 16; i++) {
                d[i] = __fsub_rn(__fadd_rn(v[i], 12582912.f), 12582912.f);   // nearest integer
                v[i] = (v[i] - d[i]) * 8.f;
            }
            *reinterpret_cast<uint2*>(dst + (size_t)q * (p.Ci / 2)) =
                make_uint2(cvt_e2m1x8(*reinterpret_cast<const float(*)[8]>(&d[0])),
                           cvt_e2m1x8(*reinterpret_cast<const float(*)[8]>(&d[8])));
        }
        // one 32-bit word of scales per column and 64-channel block, the same for all of the row's columns
        const unsigned mask = groups - (g - lane) >= 32 ? 0xffffffffu : 0xffffu;
        uint32_t word = code << (8 * (lane & 3));
        word |= __shfl_xor_sync(mask, word, 1);
        word |= __shfl_xor_sync(mask, word, 2);
        for (int q = lane & 3; q < kDigits; q += 4) {
            const int n = n0 + q;
            *reinterpret_cast<uint32_t*>(scales + ((size_t)(g >> 2) * p.sf_groups + (n >> 7)) * 512 + (n & 31) * 16 +
                                         ((n & 127) >> 5) * 4) = word;
        }
    }
}

template <int kNT, int kFmt>
__global__ void __launch_bounds__(kPrepThreads) k_rows_digits(RowsParams p) {
    extern __shared__ float low_sm[];   // [8 warps][16][rank]
    griddep_launch();
    if ((int)blockIdx.x < p.rows) return digits_of_row<kFmt>(p, (int)blockIdx.x);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int part = ((int)blockIdx.x - p.rows) % p.u_parts, m0 = ((int)blockIdx.x - p.rows) / p.u_parts * 16;
    const int nm = imin(16, p.rows - m0), nblk = p.Ci / 64;
    const int b0 = nblk * part / p.u_parts, b1 = nblk * (part + 1) / p.u_parts;
    if (part == 0 && m0 == 0 && tid == 0) *p.status = header_ok(p) ? 0 : kStatusBadWeight;
    float acc[kNT][4];
#pragma unroll
    for (int n = 0; n < kNT; n++)
#pragma unroll
        for (int i = 0; i < 4; i++) acc[n][i] = 0.f;
    for (int b = b0 + warp; b < b1; b += kPrepThreads / 32) {
        uint32_t xa[2][8];
        float sc[2];
        load_rows_16<kFmt>(p, m0, nm, b, g, t, xa, sc);
        lowrank_block<kNT, kFmt>(p, b, g, t, xa, sc, acc);
    }
    store_lowrank<kNT>(low_sm + warp * 16 * p.rank, p.rank, g, t, acc);
    __syncthreads();
    float* out = p.u_part + ((long long)part * p.rows + m0) * p.rank;
    for (int e = tid; e < nm * p.rank; e += kPrepThreads) {
        float s = 0.f;
        for (int w = 0; w < kPrepThreads / 32; w++) s += low_sm[w * 16 * p.rank + e];
        out[e] = s;
    }
}

// ------------------------------------------------------------------ the product

constexpr int kMainThreads = 384;               // producers of A and B, MMA, a spare warp, eight epilogue warps
constexpr int kEpiThreads = 256;
constexpr int kMaxSmem = 225 * 1024;

struct Fp4Bars {
    uint64_t fullA[kRowsStages], fullB[kRowsStages], empty[kRowsStages], accf;
    uint32_t tmem;
    int abort_flag;
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// 32 lanes x 16 bytes from shared memory to four columns of every 32-lane quadrant
__device__ __forceinline__ void tmem_cp_32x128b(uint32_t taddr, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

__device__ __forceinline__ void mma_nvfp4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
}

__global__ void __launch_bounds__(kMainThreads, 2)
    k_rows_fp4(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_s,
               const __grid_constant__ CUtensorMap tm_x, RowsParams p) {
    extern __shared__ __align__(16) uint8_t rows_smem[];
    uint8_t* sm = (uint8_t*)(((uintptr_t)rows_smem + 1023) & ~(uintptr_t)1023);
    __shared__ Fp4Bars bars;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = p.stages_a;
    const uint32_t b_bytes = (uint32_t)p.n_pad * 128u, sf_bytes = (uint32_t)p.sf_groups * 2048u;
    const uint32_t stage = kRowsCodeBytes + b_bytes + kRowsScaleBytes + sf_bytes;   // codes, digits, scales of both
    float* su = (float*)(sm + (size_t)S * stage);                     // [rows of the pass][rank]
    volatile int* abort_flag = &bars.abort_flag;
    const int split = (int)blockIdx.x, splits = (int)gridDim.x;       // the cluster spans a tile's splits
    const int o0 = (int)blockIdx.y * 128;
    const int m0 = (int)blockIdx.z * p.n_rows;
    const int nm = imin(p.n_rows, p.rows - m0);
    const int k256 = p.Ci / 256, a0 = k256 * split / splits, nA = k256 * (split + 1) / splits - a0;

    if (tid == 0) {
        for (int s = 0; s < S; s++) {
            mbar_init(&bars.fullA[s], 1);
            mbar_init(&bars.fullB[s], 1);
            mbar_init(&bars.empty[s], 1);
        }
        mbar_init(&bars.accf, 1);
        bars.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&bars.tmem, (uint32_t)p.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;

    if (warp == 0) {
        // ------------------------------------------------ codes and their scales
        if (lane == 0) {
            const int half = (o0 >> 7) & 1, blk0 = (o0 >> 8) * (p.Ci / 64) + a0 * 4;
            Ring r;
            int g = 0;
            for (; g < nA; g++, r.next(S)) {
                uint64_t* full = &bars.fullA[r.slot];
                if (g >= S && !mbar_wait(&bars.empty[r.slot], r.phase ^ 1, abort_flag, p.status, p.budget_ns)) break;
                uint8_t* dst = sm + (size_t)r.slot * stage;
                mbar_arrive_expect_tx(full, kRowsCodeBytes + kRowsScaleBytes);
                tma_load_2d(dst, &tm_w, full, (a0 + g) * 128, o0);
                // 32 lanes x 16 bytes per 64-channel block: one half of the 256-row tile
                tma_load_4d(dst + kRowsCodeBytes + b_bytes, &tm_s, full, 0, half, 0, blk0 + 4 * g);
            }
            for (int q = g > S ? g - S : 0; q < g; q++)   // every copy lands before shared memory is released
                mbar_wait(&bars.fullA[q % S], (uint32_t)(q / S) & 1, abort_flag, nullptr, p.budget_ns, false);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------ digits and their scales
        if (lane == 0) {
            griddep_wait();
            const uint8_t* sf = p.x_sf + ((size_t)blockIdx.z * (p.Ci / 64) + a0 * 4) * p.sf_groups * 512;
            Ring r;
            int g = 0;
            for (; g < nA; g++, r.next(S)) {
                uint64_t* full = &bars.fullB[r.slot];
                if (g >= S && !mbar_wait(&bars.empty[r.slot], r.phase ^ 1, abort_flag, p.status, p.budget_ns)) break;
                uint8_t* dst = sm + (size_t)r.slot * stage + kRowsCodeBytes;
                mbar_arrive_expect_tx(full, b_bytes + sf_bytes);
                tma_load_2d(dst, &tm_x, full, (a0 + g) * 128, m0 * kDigits);
                bulk_load(dst + b_bytes + kRowsScaleBytes, sf + (size_t)g * sf_bytes, sf_bytes, full);
            }
            for (int q = g > S ? g - S : 0; q < g; q++)
                mbar_wait(&bars.fullB[q % S], (uint32_t)(q / S) & 1, abort_flag, nullptr, p.budget_ns, false);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMAs (one elected lane; the warp's control flow is uniform)
        const uint32_t idesc = idesc_nvfp4(128, p.n_pad);
        const bool wide = p.sf_groups == 2;                       // more than 128 columns: eight scale columns a block
        const uint32_t sf_cols = wide ? 48 : 32;                  // a stage's scale columns: 16 of A, 16 or 32 of B
        const uint32_t base = smem_u32(sm);
        Ring r;
        for (int g = 0; g < nA; g++, r.next(S)) {
            if (!warp_wait(&bars.fullA[r.slot], r.phase, abort_flag, p.status, p.budget_ns)) break;
            if (!warp_wait(&bars.fullB[r.slot], r.phase, abort_flag, p.status, p.budget_ns)) break;
            tc_fence_after();
            const uint32_t sa = base + (uint32_t)r.slot * stage;
            const uint64_t ad = desc_k_sw128(sa), bd = desc_k_sw128(sa + kRowsCodeBytes);
            const uint64_t fa = smem_desc(sa + kRowsCodeBytes + b_bytes, 128, 128, 0);
            const uint64_t fb = fa + (kRowsScaleBytes >> 4);
            const uint32_t ta = tmem + (uint32_t)p.d_cols + (uint32_t)r.slot * sf_cols, tb = ta + 16;
            if (elect_one()) {
                // the stage's own columns: nothing still reads them, as its empty barrier was waited for
#pragma unroll
                for (int j = 0; j < 4; j++) tmem_cp_32x128b(ta + 4 * j, fa + 32 * j);
                if (!wide) {
#pragma unroll
                    for (int j = 0; j < 4; j++) tmem_cp_32x128b(tb + 4 * j, fb + 32 * j);
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        mma_nvfp4(tmem, ad + 2 * j, bd + 2 * j, idesc, ta + 4 * j, tb + 4 * j, (g | j) != 0);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; j++) tmem_cp_32x128b(tb + 4 * j, fb + 32 * j);
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        mma_nvfp4(tmem, ad + 2 * j, bd + 2 * j, idesc, ta + 4 * j, tb + 8 * j, (g | j) != 0);
                }
                tc_commit(&bars.empty[r.slot]);
            }
            __syncwarp();
        }
        if (elect_one()) {
            tc_commit(&bars.accf);
            mbar_wait(&bars.accf, 0, abort_flag, nullptr, p.budget_ns, false);   // no MMA runs past this point
        }
        __syncwarp();
    }

    // ---------------------------------------------------- epilogue
    const int quad = warp & 3, group = (warp - 4) >> 2, row = quad * 32 + lane, et = tid - 128;
    const PackedHeader* hdr = reinterpret_cast<const PackedHeader*>(p.packed_w);
    const float S_W = hdr->S_W;
    const int r2 = p.rank / 2;
    bool done = true, ok = true;
    float bv = 0.f;
    if (warp >= 4) {
        ok = header_ok(p);
        if (hdr->flags & kPackedHasBias) bv = *(const float*)(p.packed_w + p.off_bias + 4ll * (o0 + row));
        griddep_wait();   // the rows' factors and U come from k_rows_digits
        for (int e = et; e < nm * p.rank; e += kEpiThreads) {
            float s = 0.f;
            for (int c = 0; c < p.u_parts; c++) s += p.u_part[((long long)c * p.rows + m0) * p.rank + e];
            if (p.x_format == DQ_ROWS_E4M3) s *= p.x_scales[m0 + e / p.rank];
            su[e] = s;
        }
        bar_sync(1, kEpiThreads);
        if (lane == 0) done = mbar_wait(&bars.accf, 0, abort_flag, p.status, p.budget_ns);
        done = __shfl_sync(0xffffffffu, done, 0);
        tc_fence_after();
    }
    const uint32_t* l2 = reinterpret_cast<const uint32_t*>(p.l2 + (size_t)(o0 + row) * p.slab);
    // Y of this thread's output channel for the rows m + i * step (i < cnt <= 8) with main sums v
    auto finish = [&](int m, int step, int cnt, const float (&v)[8]) {
        float low[8];
#pragma unroll
        for (int i = 0; i < 8; i++) low[i] = 0.f;
        for (int j = 0; j < r2; j += 4) {
            const uint4 w = *reinterpret_cast<const uint4*>(l2 + j);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 8; i++) {
                if (i < cnt) {
                    const float4* u = reinterpret_cast<const float4*>(su + (m + i * step) * p.rank + 2 * j);
                    const float4 u0 = u[0], u1 = u[1];
                    low[i] = fmaf(u0.x, bf16_lo(ww[0]), low[i]);
                    low[i] = fmaf(u0.y, bf16_hi(ww[0]), low[i]);
                    low[i] = fmaf(u0.z, bf16_lo(ww[1]), low[i]);
                    low[i] = fmaf(u0.w, bf16_hi(ww[1]), low[i]);
                    low[i] = fmaf(u1.x, bf16_lo(ww[2]), low[i]);
                    low[i] = fmaf(u1.y, bf16_hi(ww[2]), low[i]);
                    low[i] = fmaf(u1.z, bf16_lo(ww[3]), low[i]);
                    low[i] = fmaf(u1.w, bf16_hi(ww[3]), low[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            if (i >= cnt) break;
            const bool two = i + 1 < cnt;
            float y0 = fmaf(v[i] * S_W, p.e[m0 + m + i * step], low[i] + bv);
            float y1 = two ? fmaf(v[i + 1] * S_W, p.e[m0 + m + (i + 1) * step], low[i + 1] + bv) : 0.f;
            if (p.gelu) f2_unpack(gelu_erf2(f2_pack(y0, y1)), y0, y1);
            uint16_t* dst = p.y + (long long)(m0 + m + i * step) * p.y_stride + o0 + row;
            dst[0] = f32_to_bf16_rn(y0);
            if (two) dst[(long long)step * p.y_stride] = f32_to_bf16_rn(y1);
        }
    };
    // main sums of the rows 8 b to 8 b + 7: their digits' columns with weights 8^-p
    auto columns = [&](int b, float (&v)[8]) {
        uint32_t acc[48];
#pragma unroll
        for (int c = 0; c < 48; c += 16)
            tmem_ld_x16(tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(48 * b + c), *reinterpret_cast<uint32_t(*)[16]>(&acc[c]));
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; i++) {
            v[i] = __uint_as_float(acc[kDigits * i + kDigits - 1]);
#pragma unroll
            for (int q = kDigits - 2; q >= 0; q--) v[i] = fmaf(v[i], 0.125f, __uint_as_float(acc[kDigits * i + q]));
        }
    };
    if (splits == 1) {
        if (warp >= 4 && done && ok) {
            for (int b = group; 8 * b < nm; b += 2) {
                float v[8];
                columns(b, v);
                finish(8 * b, 1, imin(8, nm - 8 * b), v);
            }
        }
    } else {
        // The parts of a tile: CTA r of the cluster sums, in rank order, the rows m with m % splits = r.  The
        // buffer takes the operand ring's place, so every CTA of the cluster is past its MMAs first.
        __syncwarp();
        cluster_sync();
        float* red = (float*)sm;   // [source CTA][row / splits][128 output channels]
        const int own = (nm + splits - 1) / splits;
        if (warp >= 4 && done) {
            for (int b = group; 8 * b < nm; b += 2) {
                float v[8];
                columns(b, v);
                int dst = (8 * b) % splits, at = (8 * b) / splits;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    if (8 * b + i < nm)
                        st_dsmem_f32(mapa_shared(smem_u32(&red[(split * own + at) * 128 + row]), (uint32_t)dst), v[i]);
                    if (++dst == splits) dst = 0, at++;
                }
            }
        }
        __syncwarp();
        cluster_sync();
        if (warp >= 4 && done && ok) {
            const int mine = split < nm ? (nm - split + splits - 1) / splits : 0;   // rows split, split + splits, ...
            for (int i0 = 8 * group; i0 < mine; i0 += 16) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    v[i] = 0.f;
                    if (i0 + i < mine)
                        for (int q = 0; q < splits; q++) v[i] += red[(q * own + i0 + i) * 128 + row];
                }
                finish(split + i0 * splits, splits, imin(8, mine - i0), v);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, (uint32_t)p.tmem_cols);
    }
}

template <int kNT>
cudaError_t launch_digits(const RowsParams& p, cudaStream_t st) {
    const size_t smem = (size_t)(kPrepThreads / 32) * 16 * p.rank * 4;
    const unsigned grid = (unsigned)(p.rows + p.u_parts * cdiv(p.rows, 16));
    auto go = [&](auto kernel) {
        if (smem > 48 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
        }
        kernel<<<grid, kPrepThreads, smem, st>>>(p);
        return cudaGetLastError();
    };
    if (p.x_format == DQ_ROWS_BF16) return go(k_rows_digits<kNT, DQ_ROWS_BF16>);
    if (p.x_format == DQ_ROWS_E4M3) return go(k_rows_digits<kNT, DQ_ROWS_E4M3>);
    return go(k_rows_digits<kNT, DQ_ROWS_E4M3_GROUP64>);
}

}  // namespace

// How the product of `rows` rows is cut (RowsParams' fields from n_rows on).
void rows_fp4_plan(RowsParams& p) {
    const int passes = (int)cdiv(p.rows, kRowsPass);
    p.n_rows = (int)cdiv(p.rows, passes);
    p.passes = (int)cdiv(p.rows, p.n_rows);
    p.n_pad = (int)cdiv(p.n_rows * kDigits, 8) * 8;
    p.sf_groups = p.n_pad > 128 ? 2 : 1;
    // Up to 16 rows two CTAs share an SM (256 tensor-memory columns and at most 113 KB each).  Each
    // takes more than a third of the SM's shared memory, so that a third CTA never waits there for
    // tensor memory while its cluster waits for it.
    const bool small = p.n_rows <= 16;
    p.d_cols = (int)cdiv(p.n_rows, 8) * 48;
    p.tmem_cols = small ? 256 : 512;
    const int stage = (int)(kRowsCodeBytes + kRowsScaleBytes) + p.n_pad * 128 + p.sf_groups * 2048;
    const int extra = p.n_rows * p.rank * 4 + 1024, room = (small ? 111 * 1024 : kMaxSmem) - extra;
    const int by_tmem = (p.tmem_cols - p.d_cols) / (p.sf_groups == 2 ? 48 : 32);
    p.stages_a = imin(imin(kRowsStages, room / stage), by_tmem);
    p.smem = p.stages_a * stage + extra;
    if (p.smem < 80 * 1024) p.smem = 80 * 1024;
    // as many parts of the channels as still let every CTA be resident at once
    const int tiles = p.Co / 128 * p.passes, places = small ? 296 : 148;
    p.splits = 1;
    while (p.splits < 8 && tiles * p.splits * 2 <= places && p.splits * 2 <= p.Ci / 256) p.splits *= 2;
}

cudaError_t launch_rows_fp4(const CUtensorMap& tm_w, const CUtensorMap& tm_s, const CUtensorMap& tm_x, const RowsParams& p,
                            cudaStream_t st) {
    cudaError_t e = p.rank <= 16   ? launch_digits<2>(p, st)
                    : p.rank <= 32 ? launch_digits<4>(p, st)
                    : p.rank <= 64 ? launch_digits<8>(p, st)
                                   : launch_digits<16>(p, st);
    if (e != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(k_rows_fp4, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)p.splits, (unsigned)(p.Co / 128), (unsigned)p.passes);
    cfg.blockDim = dim3(kMainThreads);
    cfg.dynamicSmemBytes = (size_t)p.smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_rows_fp4, tm_w, tm_s, tm_x, p);
}

}  // namespace dq
