// The product of few rows with a packed 4-bit weight on the block-scaled FP4
// tensor cores (dq_rows_forward; dq_rows.cu has the form for more rows).
//
// Few rows leave the weight's bytes as the bound, and decoding codes costs more
// time than reading them.  Here they are not decoded: codes and group scales are
// the A operand of kind::mxf4nvf4 as they lie in the packed weight, and a row of X
// is written in the same format as kDigits = 8 FP4 digits a value,
//   x = 2^(e-1) sum_p 8^-p d_p + r,   d_p in {-4, ..., 4},  |r| <= 2^(e-23),
// with 2^e <= max |x| < 2^(e+1) over the row and d_p the nearest integer to what
// the digits before it leave: 24 bits of the row's largest value, what an fp32 sum
// over the row keeps of it.  Each digit is a column of the MMA (the B scales are 1)
// and the epilogue sums a row's columns with their weights 8^-p in fp32.
//
//   k_rows_digits   digits and 2^(e-1) per row; beside it U = xv L1 in up to 16
//                   partial sums over the channels (mma.sync)
//   k_rows_fp4      128 output channels (the MMA's M) times up to 32 rows (256
//                   columns) per CTA.  One warp keeps codes and scales in flight,
//                   one the digits, one issues scale copies and MMAs, eight form
//                   U L2 meanwhile and then the output.  When the tiles alone do
//                   not fill the GPU a cluster splits the channels and sums its
//                   parts in rank order through distributed shared memory.  The
//                   loads of the weight do not wait for k_rows_digits
//                   (programmatic launch).
#include "../../include/deltaquant.h"
#include "dq_common.h"
#include "dq_internal.h"
#include "dq_ptx.cuh"
#include "dq_rows.cuh"

#include <atomic>

namespace dq {

namespace {

constexpr int kDigits = kRowsDigits;

// ------------------------------------------------------------------ rows -> digits, and U

constexpr int kPrepThreads = 256;

// The values of eight consecutive channels from c on of row m
template <int kFmt>
__device__ __forceinline__ void load_values8(const RowsParams& p, int m, int c, float (&v)[8]) {
    const long long off = (long long)m * p.x_stride + c;
    if (kFmt == DQ_ROWS_BF16) {
        const uint4 a = *reinterpret_cast<const uint4*>((const uint16_t*)p.x + off);
        const uint32_t r[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; i++) v[2 * i] = bf16_lo(r[i]), v[2 * i + 1] = bf16_hi(r[i]);
    } else {
        const uint2 a = *reinterpret_cast<const uint2*>((const uint8_t*)p.x + off);
        const uint32_t r[2] = {a.x, a.y};
        const float s = kFmt == DQ_ROWS_E4M3_GROUP64 ? p.x_scales[(long long)m * (p.Ci / 64) + c / 64] : 1.f;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            f16x2_values(e4m3x2_to_f16x2(r[i / 2] >> (16 * (i & 1))), v[2 * i], v[2 * i + 1]);
            if (kFmt == DQ_ROWS_E4M3_GROUP64) v[2 * i] *= s, v[2 * i + 1] *= s;
        }
    }
}

// Digits of the channels 2048 part to 2048 part + 2047 of row m (each CTA of a row finds the row's
// largest magnitude for itself: a second read of at most 28 KB, from L2, instead of a hand-off).
template <int kFmt>
__device__ __forceinline__ void digits_of_row(const RowsParams& p, int m, int part) {
    __shared__ float sh[kPrepThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, c = (part * kPrepThreads + tid) * 8;
    float v[8], am = 0.f;
    for (int i = tid * 8; i < p.Ci; i += kPrepThreads * 8) {
        load_values8<kFmt>(p, m, i, v);
#pragma unroll
        for (int e = 0; e < 8; e++) am = max_nan(am, fabsf(v[e]));
    }
    if (c < p.Ci) load_values8<kFmt>(p, m, c, v);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
    if (lane == 0) sh[tid >> 5] = am;
    __syncthreads();
    am = sh[0];
#pragma unroll
    for (int w = 1; w < kPrepThreads / 32; w++) am = max_nan(am, sh[w]);
    const bool finite = am < __int_as_float(0x7F800000);
    const int eb = (int)((__float_as_uint(am) >> 23) & 255);
    const int k = (eb ? eb - 127 : -126) - 1;       // the first digit's unit 2^k; |x 2^-k| < 4
    if (part == 0 && tid == 0) {
        float E = k >= -126 ? pow2i(k) : __int_as_float(1 << (k + 149));
        if (kFmt == DQ_ROWS_E4M3) E *= p.x_scales[m];
        p.e[m] = finite ? E : __int_as_float(0x7FC00000);   // a NaN or an infinity: NaN all over the row
    }
    if (c >= p.Ci) return;
    const int h = -k / 2;                            // two exact steps (k in [-127, 126])
    const float f0 = pow2i(h), f1 = pow2i(-k - h);
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = finite ? v[i] * f0 * f1 : 0.f;
    uint8_t* dst = (uint8_t*)p.xh + (size_t)m * kDigits * (p.Ci / 2) + c / 2;
#pragma unroll
    for (int q = 0; q < kDigits; q++) {
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            d[i] = __fsub_rn(__fadd_rn(v[i], 12582912.f), 12582912.f);   // nearest integer
            v[i] = (v[i] - d[i]) * 8.f;
        }
        *reinterpret_cast<uint32_t*>(dst + (size_t)q * (p.Ci / 2)) = cvt_e2m1x8(d);
    }
}

template <int kNT, int kFmt>
__global__ void __launch_bounds__(kPrepThreads) k_rows_digits(RowsParams p) {
    extern __shared__ float low_sm[];   // [8 warps][16][rank]
    griddep_wait();     // the launch before this one may still read the workspace, or write X
    griddep_launch();
    const int parts = (p.Ci + 2047) / 2048, block = (int)blockIdx.x;
    if (block < p.rows * parts) return digits_of_row<kFmt>(p, block / parts, block % parts);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int part = (block - p.rows * parts) % p.u_parts, m0 = (block - p.rows * parts) / p.u_parts * 16;
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
constexpr int kMaxSmem = 225 * 1024, kSmallSmem = 225 * 512;   // dynamic shared memory, one CTA or two per SM

struct Fp4Bars {
    uint64_t full[kRowsStages], empty[kRowsStages], accf;
    uint32_t tmem;
    int abort_flag;
};

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
    const uint32_t b_bytes = (uint32_t)p.n_pad * 128u;
    const uint32_t stage = kRowsCodeBytes + b_bytes + kRowsScaleBytes;   // codes, digits, the codes' scales
    float* su = (float*)(sm + (size_t)S * stage);                     // [rows of the pass][rank]: U
    float* se = su + p.n_rows * p.rank;                               // [rows of the pass]: the rows' factors
    float* slow = se + 64;                                            // [rows this CTA finishes][128]: U L2 + b
    volatile int* abort_flag = &bars.abort_flag;
    const int split = (int)blockIdx.x, splits = (int)gridDim.x;       // the cluster spans a tile's splits
    const int o0 = (int)blockIdx.y * 128;
    const int m0 = (int)blockIdx.z * p.n_rows;
    const int nm = imin(p.n_rows, p.rows - m0);
    const int k256 = p.Ci / 256, a0 = k256 * split / splits, nA = k256 * (split + 1) / splits - a0;

    if (tid == 0) {
        for (int s = 0; s < S; s++) {
            mbar_init(&bars.full[s], 2);    // both producers
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
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tm_w);
        prefetch_tmap(&tm_s);
    }
    if (warp == 2 && lane == 0) prefetch_tmap(&tm_x);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem, t_one = tmem + (uint32_t)p.d_cols, t_sf = t_one + 8;
    griddep_launch();

    if (warp == 0) {
        // ------------------------------------------------ codes and their scales
        if (lane == 0) {
            const int half = (o0 >> 7) & 1, blk0 = (o0 >> 8) * (p.Ci / 64) + a0 * 4;
            Ring r;
            int g = 0;
            for (; g < nA; g++, r.next(S)) {
                uint64_t* full = &bars.full[r.slot];
                if (g >= S && !mbar_wait(&bars.empty[r.slot], r.phase ^ 1, abort_flag, p.status, p.budget_ns)) break;
                uint8_t* dst = sm + (size_t)r.slot * stage;
                mbar_arrive_expect_tx(full, kRowsCodeBytes + kRowsScaleBytes);
                tma_load_2d(dst, &tm_w, full, (a0 + g) * 128, o0);
                // 32 lanes x 16 bytes per 64-channel block: one half of the 256-row tile
                tma_load_4d(dst + kRowsCodeBytes + b_bytes, &tm_s, full, 0, half, 0, blk0 + 4 * g);
            }
            for (int q = g > S ? g - S : 0; q < g; q++)   // every copy lands before shared memory is released
                mbar_wait(&bars.full[q % S], (uint32_t)(q / S) & 1, abort_flag, nullptr, p.budget_ns, false);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------ digits
        if (lane == 0) {
            griddep_wait();
            Ring r;
            int g = 0;
            for (; g < nA; g++, r.next(S)) {
                uint64_t* full = &bars.full[r.slot];
                if (g >= S && !mbar_wait(&bars.empty[r.slot], r.phase ^ 1, abort_flag, p.status, p.budget_ns)) break;
                mbar_arrive_expect_tx(full, b_bytes);
                tma_load_2d(sm + (size_t)r.slot * stage + kRowsCodeBytes, &tm_x, full, (a0 + g) * 128, m0 * kDigits);
            }
            for (int q = g > S ? g - S : 0; q < g; q++)
                mbar_wait(&bars.full[q % S], (uint32_t)(q / S) & 1, abort_flag, nullptr, p.budget_ns, false);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMAs (one elected lane; the warp's control flow is uniform)
        const uint32_t idesc = idesc_nvfp4(128, p.n_pad);
        const uint32_t base = smem_u32(sm);
        bar_sync(2, 32 + 128);   // the digits' scales are in tensor memory
        tc_fence_after();
        Ring r;
        uint32_t sa = base, ta = t_sf;
        for (int g = 0; g < nA; g++) {
            if (!__all_sync(0xffffffffu, mbar_wait_spin(&bars.full[r.slot], r.phase, abort_flag, p.status, p.budget_ns))) break;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t ad = desc_k_sw128(sa), bd = desc_k_sw128(sa + kRowsCodeBytes);
                const uint64_t fa = smem_desc(sa + kRowsCodeBytes + b_bytes, 128, 128, 0);
                // the stage's own columns: nothing still reads them, as its empty barrier was waited for
#pragma unroll
                for (int j = 0; j < 4; j++) tmem_cp_32x128b(ta + 4 * j, fa + 32 * j);
#pragma unroll
                for (int j = 0; j < 4; j++) mma_nvfp4(tmem, ad + 2 * j, bd + 2 * j, idesc, ta + 4 * j, t_one, (g | j) != 0);
                tc_commit(&bars.empty[r.slot]);
            }
            __syncwarp();
            sa += stage, ta += 16;
            r.next(S);
            if (r.slot == 0) sa = base, ta = t_sf;
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
    // the rows of the pass that this CTA finishes: every splits-th
    const int mine = split < nm ? (nm - split + splits - 1) / splits : 0;
    bool done = true, ok = true;
    if (warp >= 4) {
        if (warp < 8) {
            // the digits' scales: E4M3 1 in eight columns of every lane
            const uint32_t one = 0x38383838u, at = t_one + ((uint32_t)(quad * 32) << 16);
            tmem_st_x4(at, one, one, one, one);
            tmem_st_x4(at + 4, one, one, one, one);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            asm volatile("bar.arrive 2, 160;" ::: "memory");
        }
        ok = header_ok(p);
        float bv = 0.f;
        if (hdr->flags & kPackedHasBias) bv = *(const float*)(p.packed_w + p.off_bias + 4ll * (o0 + row));
        // U, the rows' factors and U L2 + b while the weight streams in
        griddep_wait();
        for (int e = et; e < nm * p.rank; e += kEpiThreads) {
            float s = 0.f;
            for (int c = 0; c < p.u_parts; c++) s += p.u_part[((long long)c * p.rows + m0) * p.rank + e];
            if (p.x_format == DQ_ROWS_E4M3) s *= p.x_scales[m0 + e / p.rank];
            su[e] = s;
        }
        if (et < nm) se[et] = p.e[m0 + et];
        bar_sync(1, kEpiThreads);
        const uint4* l2 = reinterpret_cast<const uint4*>(p.l2 + (size_t)(o0 + row) * p.slab);
        for (int i0 = 4 * group; i0 < mine; i0 += 8) {
            float low[4] = {bv, bv, bv, bv};
            for (int j = 0; j < p.rank; j += 8) {
                const uint4 w = l2[j / 8];
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (i0 + i < mine) {
                        const float4* u = reinterpret_cast<const float4*>(su + (split + (i0 + i) * splits) * p.rank + j);
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
            for (int i = 0; i < 4; i++)
                if (i0 + i < mine) slow[(i0 + i) * 128 + row] = low[i];
        }
        bar_sync(1, kEpiThreads);
        if (lane == 0) done = mbar_wait(&bars.accf, 0, abort_flag, p.status, p.budget_ns);
        done = __shfl_sync(0xffffffffu, done, 0);
        tc_fence_after();
    }
    // Y of this thread's output channel for the rows i, i + 1 of those this CTA finishes (the second where
    // it exists), from their main sums
    auto finish = [&](int i, float v0, float v1) {
        const bool two = i + 1 < mine;
        const int m = split + i * splits;
        float y0 = fmaf(v0 * S_W, se[m], slow[i * 128 + row]);
        float y1 = two ? fmaf(v1 * S_W, se[m + splits], slow[(i + 1) * 128 + row]) : 0.f;
        if (p.gelu) f2_unpack(gelu_erf2(f2_pack(y0, y1)), y0, y1);
        uint16_t* dst = p.y + (long long)(m0 + m) * p.y_stride + o0 + row;
        dst[0] = f32_to_bf16_rn(y0);
        if (two) dst[(long long)splits * p.y_stride] = f32_to_bf16_rn(y1);
    };
    // main sums of the rows 4 b to 4 b + 3: their digits' columns with weights 8^-p
    auto columns = [&](int b, float (&v)[4]) {
        uint32_t acc[32];
#pragma unroll
        for (int c = 0; c < 32; c += 16)
            tmem_ld_x16(tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(32 * b + c), *reinterpret_cast<uint32_t(*)[16]>(&acc[c]));
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[i] = __uint_as_float(acc[kDigits * i + kDigits - 1]);
#pragma unroll
            for (int q = kDigits - 2; q >= 0; q--) v[i] = fmaf(v[i], 0.125f, __uint_as_float(acc[kDigits * i + q]));
        }
    };
    if (splits == 1) {
        if (warp >= 4 && done && ok) {
            for (int b = group; 4 * b < nm; b += 2) {
                float v[4];
                columns(b, v);
                finish(4 * b, v[0], v[1]);
                if (4 * b + 2 < nm) finish(4 * b + 2, v[2], v[3]);
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
            for (int b = group; 4 * b < nm; b += 2) {
                float v[4];
                columns(b, v);
                int dst = (4 * b) % splits, at = (4 * b) / splits;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (4 * b + i < nm)
                        st_dsmem_f32(mapa_shared(smem_u32(&red[(split * own + at) * 128 + row]), (uint32_t)dst), v[i]);
                    if (++dst == splits) dst = 0, at++;
                }
            }
        }
        __syncwarp();
        cluster_sync();
        if (warp >= 4 && done && ok) {
            for (int i = 2 * group; i < mine; i += 4) {
                float v0 = 0.f, v1 = 0.f;
                for (int q = 0; q < splits; q++) {
                    v0 += red[(q * own + i) * 128 + row];
                    if (i + 1 < mine) v1 += red[(q * own + i + 1) * 128 + row];
                }
                finish(i, v0, v1);
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

// Runs `set` (a kernel's attributes) on the first call for that kernel on the current device.  Concurrent
// first calls may both run it; they set the same values.
template <typename Set>
cudaError_t once_per_device(const void* kernel, Set set) {
    constexpr int kKernels = 16, kDevices = 64;
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

template <int kNT>
cudaError_t launch_digits(const RowsParams& p, cudaStream_t st) {
    const size_t smem = (size_t)(kPrepThreads / 32) * 16 * p.rank * 4;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(p.rows * cdiv(p.Ci, 2048) + p.u_parts * cdiv(p.rows, 16)));
    cfg.blockDim = dim3(kPrepThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto go = [&](auto kernel) {
        // the product's split of the SM between L1 and shared memory: a different one would keep its CTAs
        // off an SM until this kernel's have left
        const cudaError_t e = once_per_device((const void*)kernel, [&] {
            cudaError_t e1 = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                  (kPrepThreads / 32) * 16 * 8 * kNT * 4);
            return e1 != cudaSuccess ? e1 : cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        });
        if (e != cudaSuccess) return e;
        return cudaLaunchKernelEx(&cfg, kernel, p);
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
    p.n_pad = p.n_rows * kDigits;
    // Up to 16 rows two CTAs share an SM (256 tensor-memory columns and at most 113 KB each).  Each
    // takes more than a third of the SM's shared memory, so that a third CTA never waits there for
    // tensor memory while its cluster waits for it.
    const bool small = p.n_rows <= 16;
    p.d_cols = (int)cdiv(p.n_pad, 32) * 32;
    p.tmem_cols = small ? 256 : 512;
    const int stage = (int)(kRowsCodeBytes + kRowsScaleBytes) + p.n_pad * 128;
    // as many parts of the channels as still let every CTA be resident at once
    const int tiles = p.Co / 128 * p.passes, places = small ? 296 : 148;
    p.splits = 1;
    while (p.splits < 8 && tiles * p.splits * 2 <= places && p.splits * 2 <= p.Ci / 256) p.splits *= 2;
    const int extra = (p.n_rows * p.rank + 64 + (int)cdiv(p.n_rows, p.splits) * 128) * 4 + 1024;
    const int room = (small ? kSmallSmem : kMaxSmem) - extra;
    p.stages_a = imin(imin(kRowsStages, room / stage), (p.tmem_cols - p.d_cols - 8) / 16);
    p.smem = p.stages_a * stage + extra;
    if (p.smem < 80 * 1024) p.smem = 80 * 1024;
}

cudaError_t launch_rows_fp4(const CUtensorMap& tm_w, const CUtensorMap& tm_s, const CUtensorMap& tm_x, const RowsParams& p,
                            cudaStream_t st) {
    cudaError_t e = p.rank <= 16   ? launch_digits<2>(p, st)
                    : p.rank <= 32 ? launch_digits<4>(p, st)
                    : p.rank <= 64 ? launch_digits<8>(p, st)
                                   : launch_digits<16>(p, st);
    if (e != cudaSuccess) return e;
    e = once_per_device((const void*)k_rows_fp4, [] {
        return cudaFuncSetAttribute(k_rows_fp4, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    });
    if (e != cudaSuccess) return e;
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
