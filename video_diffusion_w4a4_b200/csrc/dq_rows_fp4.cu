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
// The low-rank factor is BF16 K steps of the same warp into columns of its own
// (U as hi + lo times L2, one column a row).
//
//   k_rows_fp4   128 output channels (the MMA's M) times up to 32 rows (256
//                columns) per CTA.  One warp keeps codes and scales in flight, one
//                the digits, one issues scale copies and MMAs, eight write the
//                output.  When the tiles alone do not fill the GPU a cluster splits
//                the channels and sums its parts in rank order through distributed
//                shared memory.  The loads of the weight do not wait for
//                k_rows_prepare (programmatic launch).
#include "../../include/deltaquant.h"
#include "dq_common.h"
#include "dq_internal.h"
#include "dq_ptx.cuh"
#include "dq_rows.cuh"

namespace dq {

namespace {

constexpr int kDigits = kRowsDigits;

// ------------------------------------------------------------------ the product

constexpr int kMainThreads = 384;               // producers of A and B, MMA, a spare warp, eight epilogue warps
constexpr int kEpiThreads = 256;
constexpr int kMaxSmem = 225 * 1024, kSmallSmem = 112 * 1024;   // dynamic shared memory, one CTA or two per SM

constexpr int kOwnTurns = 8;                    // pieces of eight channels a thread holds (own digits)

struct Fp4Bars {
    uint64_t full[kRowsStages], empty[kRowsStages], accf, digits[kOwnTurns];
    float e[kRowsPass];   // the rows' factors
    float amax[8];        // own digits: each warp's part of its row's largest magnitude
    uint32_t tmem;
    int abort_flag;
};

// Each thread of the warp reads four consecutive 32-bit columns of its lane.
__device__ __forceinline__ void tmem_ld_x4(uint32_t taddr, uint32_t (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr)
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

// Own digits (at most kRowsOwn rows): the epilogue warps, idle while the weight streams in, write the digits of
// this CTA's channels into shared memory as the MMA reads them, with the power of two of the rows' values in these
// channels alone.  Each row takes own_warps(rows) warps, which hold all its values from one read and write the
// digits 256 channels a warp at a time, each such turn with a barrier of its own for the MMAs.
__host__ __device__ constexpr int own_warps(int rows) { return rows == 1 ? 8 : rows == 2 ? 4 : rows <= 4 ? 2 : 1; }

template <int kFmt>
__device__ __forceinline__ void write_own_digits(const RowsParams& p, Fp4Bars& bars, uint8_t* dst, int c0, int channels) {
    const int ew = (int)(threadIdx.x >> 5) - 4, lane = threadIdx.x & 31;
    const int per = own_warps(p.rows), m = ew / per, part = ew % per, first = (part * 32 + lane) * 8;
    Raw8<kFmt> raw[kOwnTurns];
    float am = 0.f;
#pragma unroll
    for (int i = 0; i < kOwnTurns; i++) {
        raw[i] = {};
        if (m < p.rows && first + i * per * 256 < channels) raw[i] = load_raw8<kFmt>(p, m, c0 + first + i * per * 256);
    }
#pragma unroll
    for (int i = 0; i < kOwnTurns; i++) am = max_nan(am, amax8<kFmt>(raw[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
    if (lane == 0) bars.amax[ew] = am;
    bar_sync(1, kEpiThreads);
    for (int i = 0; i < per; i++) am = max_nan(am, bars.amax[m * per + i]);
    const bool finite = finite_row(am);
    const int k = row_unit<kFmt, true>(am);
    if (m < p.rows && part == 0 && lane == 0) {
        float E = k >= -126 ? pow2i(k) : __int_as_float(1 << (k + 149));
        if (kFmt == DQ_ROWS_E4M3) E *= p.x_scales[m];
        bars.e[m] = finite ? E : __int_as_float(0x7FC00000);
    }
    const Scale2 s = inv_scale(k);
#pragma unroll
    for (int i = 0; i < kOwnTurns; i++) {
        const int c = first + i * per * 256;
        if (i * per * 256 < channels) {
            if (m < p.rows && c < channels) {
                float v[8];
                uint64_t v2[4];
                values8<kFmt>(raw[i], v);
                scaled_pairs(v, s, finite, v2);
                // column 8 m + q of the 256-channel stage c / 256: row 8 m + q of 128 bytes, its 16-byte pieces
                // permuted by the row's low bits (128-byte swizzle)
                uint8_t* row = dst + (size_t)(c >> 8) * p.n_pad * 128 + m * 1024 + ((c >> 1) & 15);
                const int piece = (c >> 5) & 7;
#pragma unroll
                for (int q = 0; q < kDigits; q++)
                    *reinterpret_cast<uint32_t*>(row + q * 128 + ((piece ^ q) << 4)) = next_digits8(v2);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the MMA reads them
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.digits[i]);
        }
    }
    bar_sync(1, kEpiThreads);   // the factors, for every epilogue warp
}

__global__ void __launch_bounds__(kMainThreads, 2)
    k_rows_fp4(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_s,
               const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_l2,
               const __grid_constant__ CUtensorMap tm_u, RowsParams p) {
    extern __shared__ __align__(16) uint8_t rows_smem[];
    uint8_t* sm = (uint8_t*)(((uintptr_t)rows_smem + 1023) & ~(uintptr_t)1023);
    __shared__ Fp4Bars bars;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = p.stages_a;
    const bool own = p.own_digits != 0;
    const uint32_t b_all = (uint32_t)p.n_pad * 128u, b_bytes = own ? 0u : b_all;   // digits of a stage; in the ring
    const uint32_t stage = kRowsCodeBytes + b_bytes + kRowsScaleBytes;   // codes, digits, the codes' scales
    volatile int* abort_flag = &bars.abort_flag;
    const int split = (int)blockIdx.x, splits = (int)gridDim.x;       // the cluster spans a tile's splits
    const int o0 = (int)blockIdx.y * 128;
    const int m0 = (int)blockIdx.z * p.n_rows;
    const int nm = imin(p.n_rows, p.rows - m0);
    const int k256 = p.Ci / 256, a0 = k256 * split / splits, nA = k256 * (split + 1) / splits - a0;
    const int total = nA + (split == 0 ? p.slab / 64 : 0);           // stages: the weight's, then the low-rank factor's
    const uint32_t n16 = (uint32_t)(p.n_rows + 15) & ~15u;
    uint8_t* digits = sm + (size_t)S * stage;                         // own digits: [stage][column][128 bytes]

    if (tid == 0) {
        for (int s = 0; s < S; s++) {
            mbar_init(&bars.full[s], own ? 1 : 2);   // one producer, or both
            mbar_init(&bars.empty[s], 1);
        }
        mbar_init(&bars.accf, 1);
        for (int i = 0; i < kOwnTurns; i++) mbar_init(&bars.digits[i], kEpiThreads / 32);
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
    if (warp == 2 && lane == 0) prefetch_tmap(&tm_x), prefetch_tmap(&tm_u), prefetch_tmap(&tm_l2);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem, t_low = tmem + (uint32_t)p.d_cols, t_one = t_low + n16, t_sf = t_one + 8;
    griddep_launch();

    if (warp == 0) {
        // ------------------------------------------------ codes and their scales
        if (lane == 0) {
            const int half = (o0 >> 7) & 1, blk0 = (o0 >> 8) * (p.Ci / 64) + a0 * 4;
            Ring r;
            int g = 0;
            for (; g < total; g++, r.next(S)) {
                uint64_t* full = &bars.full[r.slot];
                if (g >= S && !mbar_wait(&bars.empty[r.slot], r.phase ^ 1, abort_flag, p.status, p.budget_ns)) break;
                uint8_t* dst = sm + (size_t)r.slot * stage;
                if (g < nA) {
                    mbar_arrive_expect_tx(full, kRowsCodeBytes + kRowsScaleBytes);
                    tma_load_2d(dst, &tm_w, full, (a0 + g) * 128, o0);
                    // 32 lanes x 16 bytes per 64-channel block: one half of the 256-row tile
                    tma_load_4d(dst + kRowsCodeBytes + b_bytes, &tm_s, full, 0, half, 0, blk0 + 4 * g);
                } else if (!own) {
                    mbar_arrive_expect_tx(full, kRowsCodeBytes);
                    tma_load_2d(dst, &tm_l2, full, (g - nA) * 64, o0);
                } else {
                    if (g == nA) griddep_wait();   // U comes from k_rows_prepare
                    mbar_arrive_expect_tx(full, kRowsCodeBytes + n16 * 128);
                    tma_load_2d(dst, &tm_l2, full, (g - nA) * 64, o0);
                    tma_load_2d(dst + kRowsCodeBytes, &tm_u, full, (g - nA) * 64, m0);
                }
            }
            for (int q = g > S ? g - S : 0; q < g; q++)   // every copy lands before shared memory is released
                mbar_wait(&bars.full[q % S], (uint32_t)(q / S) & 1, abort_flag, nullptr, p.budget_ns, false);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------ digits, then U
        if (lane == 0 && !own) {
            griddep_wait();
            Ring r;
            int g = 0;
            for (; g < total; g++, r.next(S)) {
                uint64_t* full = &bars.full[r.slot];
                if (g >= S && !mbar_wait(&bars.empty[r.slot], r.phase ^ 1, abort_flag, p.status, p.budget_ns)) break;
                uint8_t* dst = sm + (size_t)r.slot * stage + kRowsCodeBytes;
                if (g < nA) {
                    mbar_arrive_expect_tx(full, b_bytes);
                    tma_load_2d(dst, &tm_x, full, (a0 + g) * 128, m0 * kDigits);
                } else {
                    mbar_arrive_expect_tx(full, n16 * 128);   // within the digits' and the scales' places
                    tma_load_2d(dst, &tm_u, full, (g - nA) * 64, m0);
                }
            }
            for (int q = g > S ? g - S : 0; q < g; q++)
                mbar_wait(&bars.full[q % S], (uint32_t)(q / S) & 1, abort_flag, nullptr, p.budget_ns, false);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMAs (one elected lane; the warp's control flow is uniform)
        const uint32_t idesc = idesc_nvfp4(128, p.n_pad), id_low = idesc_bf16(128, (int)n16);
        const uint32_t base = smem_u32(sm);
        bar_sync(2, 32 + 128);   // the digits' scales are in tensor memory
        tc_fence_after();
        Ring r;
        uint32_t sa = base, ta = t_sf, sb = own ? smem_u32(digits) : base + kRowsCodeBytes;
        const uint32_t b_step = own ? b_all : stage;
        int turn = 0, left = 0;                          // own digits: stages until the next turn's barrier
        for (int g = 0; g < total; g++) {
            if (own && g < nA && left-- == 0) {
                if (!__all_sync(0xffffffffu, mbar_wait_spin(&bars.digits[turn], 0, abort_flag, p.status, p.budget_ns))) break;
                turn++;
                left = own_warps(p.rows) - 1;
            }
            if (!__all_sync(0xffffffffu, mbar_wait_spin(&bars.full[r.slot], r.phase, abort_flag, p.status, p.budget_ns))) break;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t ad = desc_k_sw128(sa);
                if (g < nA) {
                    const uint64_t bd = desc_k_sw128(sb);
                    const uint64_t fa = smem_desc(sa + kRowsCodeBytes + b_bytes, 128, 128, 0);
                    // the stage's own columns: nothing still reads them, as its empty barrier was waited for
#pragma unroll
                    for (int j = 0; j < 4; j++) tmem_cp_32x128b(ta + 4 * j, fa + 32 * j);
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        mma_nvfp4(tmem, ad + 2 * j, bd + 2 * j, idesc, ta + 4 * j, t_one, (g | j) != 0);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; j++) mma_bf16(t_low, ad + 2 * j, desc_k_sw128(sa + kRowsCodeBytes) + 2 * j, id_low, (g > nA || j) ? 1u : 0u);
                }
                tc_commit(&bars.empty[r.slot]);
            }
            __syncwarp();
            sa += stage, ta += 16, sb += b_step;
            r.next(S);
            if (r.slot == 0) {
                sa = base, ta = t_sf;
                if (!own) sb = base + kRowsCodeBytes;
            }
        }
        if (elect_one()) {
            tc_commit(&bars.accf);
            mbar_wait(&bars.accf, 0, abort_flag, nullptr, p.budget_ns, false);   // no MMA runs past this point
        }
        __syncwarp();
    }

    // ---------------------------------------------------- epilogue
    const int quad = warp & 3, group = (warp - 4) >> 2, row = quad * 32 + lane, et = tid - 128;
    const uint32_t trow = (uint32_t)(quad * 32) << 16;
    const PackedHeader* hdr = reinterpret_cast<const PackedHeader*>(p.packed_w);
    bool done = true, ok = true;
    float bv = 0.f, S_W = 0.f;
    if (warp >= 4) {
        if (warp < 8) {
            // the digits' scales: E4M3 1 in eight columns of every lane
            const uint32_t one = 0x38383838u;
            tmem_st_x4(t_one + trow, one, one, one, one);
            tmem_st_x4(t_one + trow + 4, one, one, one, one);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            asm volatile("bar.arrive 2, 160;" ::: "memory");
        }
        if (own) {
            uint8_t* dst = digits;
            if (p.x_format == DQ_ROWS_BF16)
                write_own_digits<DQ_ROWS_BF16>(p, bars, dst, a0 * 256, nA * 256);
            else if (p.x_format == DQ_ROWS_E4M3)
                write_own_digits<DQ_ROWS_E4M3>(p, bars, dst, a0 * 256, nA * 256);
            else
                write_own_digits<DQ_ROWS_E4M3_GROUP64>(p, bars, dst, a0 * 256, nA * 256);
        } else {
            griddep_wait();   // the rows' factors come from k_rows_prepare
            if (et < nm) bars.e[et] = p.e[m0 + et];
            bar_sync(1, kEpiThreads);
        }
        ok = header_ok(p);
        S_W = hdr->S_W;
        if (hdr->flags & kPackedHasBias) bv = *(const float*)(p.packed_w + p.off_bias + 4ll * (o0 + row));
        if (lane == 0) done = mbar_wait(&bars.accf, 0, abort_flag, p.status, p.budget_ns);
        done = __shfl_sync(0xffffffffu, done, 0);
        tc_fence_after();
    }
    // This CTA's part of the rows 4 b to 4 b + 3 for the thread's output channel: the digits' columns with
    // weights 8^-p, times S_W and the row's factor, and U L2 where this CTA has it
    auto parts_of = [&](int b, float (&v)[4]) {
        uint32_t acc[32], low[4];
#pragma unroll
        for (int c = 0; c < 32; c += 16) tmem_ld_x16(tmem + trow + (uint32_t)(32 * b + c), *reinterpret_cast<uint32_t(*)[16]>(&acc[c]));
        if (split == 0) tmem_ld_x4(t_low + trow + (uint32_t)(4 * b), low);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[i] = __uint_as_float(acc[kDigits * i + kDigits - 1]);
#pragma unroll
            for (int q = kDigits - 2; q >= 0; q--) v[i] = fmaf(v[i], 0.125f, __uint_as_float(acc[kDigits * i + q]));
            v[i] = fmaf(v[i] * S_W, bars.e[imin(4 * b + i, nm - 1)], split == 0 ? __uint_as_float(low[i]) : 0.f);
        }
    };
    // Y of the thread's output channel for the row m of the pass and the row m + step where `two` is set
    auto finish = [&](int m, int step, bool two, float y0, float y1) {
        y0 += bv, y1 += bv;
        if (p.gelu) f2_unpack(gelu_erf2(f2_pack(y0, y1)), y0, y1);
        uint16_t* dst = p.y + (long long)(m0 + m) * p.y_stride + o0 + row;
        dst[0] = f32_to_bf16_rn(y0);
        if (two) dst[(long long)step * p.y_stride] = f32_to_bf16_rn(y1);
    };
    if (splits == 1) {
        if (warp >= 4 && done && ok) {
            for (int b = group; 4 * b < nm; b += 2) {
                float v[4];
                parts_of(b, v);
                finish(4 * b, 1, 4 * b + 1 < nm, v[0], v[1]);
                if (4 * b + 2 < nm) finish(4 * b + 2, 1, 4 * b + 3 < nm, v[2], v[3]);
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
                parts_of(b, v);
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
            const int mine = split < nm ? (nm - split + splits - 1) / splits : 0;   // rows split, split + splits, ...
            for (int i = 2 * group; i < mine; i += 4) {
                float v0 = 0.f, v1 = 0.f;
                for (int q = 0; q < splits; q++) {
                    v0 += red[(q * own + i) * 128 + row];
                    if (i + 1 < mine) v1 += red[(q * own + i + 1) * 128 + row];
                }
                finish(split + i * splits, splits, i + 1 < mine, v0, v1);
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

}  // namespace

namespace {

cudaError_t set_attributes() {
    return once_per_device((const void*)k_rows_fp4, [] {
        return cudaFuncSetAttribute(k_rows_fp4, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    });
}

// Clusters of `splits` CTAs that fit on the current device at once, asked once per device and configuration.
cudaError_t resident_clusters(bool small, int splits, int* clusters) {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][2][9];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    std::atomic<int>& k = known[dev][small][splits];
    if ((*clusters = k.load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    if ((e = set_attributes()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)splits, 1024);
    cfg.blockDim = dim3(kMainThreads);
    cfg.dynamicSmemBytes = small ? kSmallSmem : kMaxSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaOccupancyMaxActiveClusters(clusters, k_rows_fp4, &cfg)) != cudaSuccess) return e;
    k.store(*clusters, std::memory_order_relaxed);
    return cudaSuccess;
}

}  // namespace

// How the product of `rows` rows is cut (RowsParams' fields from n_rows on).
cudaError_t rows_fp4_plan(RowsParams& p) {
    const int passes = (int)cdiv(p.rows, kRowsPass);
    p.n_rows = (int)cdiv(p.rows, passes);
    p.passes = (int)cdiv(p.rows, p.n_rows);
    p.n_pad = p.n_rows * kDigits;
    p.d_cols = (int)cdiv(p.n_pad, 32) * 32;
    const int tiles = p.Co / 128 * p.passes, k256 = p.Ci / 256, low = p.slab / 64;
    const int stage_w = (int)(kRowsCodeBytes + kRowsScaleBytes), digits = p.n_pad * 128;
    // Up to 16 rows two CTAs share an SM (256 tensor-memory columns and half the shared memory each; a third
    // never fits, so none waits there for tensor memory while its cluster waits for it).  A cluster
    // splits the channels as far as all CTAs are still resident at once.  Rows up to kRowsOwn get their digits
    // from the product itself if those and a ring of enough stages fit, on half an SM or else on a whole one.
    for (int attempt = 0; attempt < 4; attempt++) {
        const bool own = attempt < 2, small = attempt % 2 == 0;
        if ((own && p.rows > kRowsOwn) || (small && p.n_rows > 16)) continue;
        p.splits = 1;
        const int tries[] = {8, 6, 4, 3, 2};
        for (int s : tries) {
            int clusters = 0;
            cudaError_t e = s <= k256 ? resident_clusters(small, s, &clusters) : cudaSuccess;
            if (e != cudaSuccess) return e;
            if (s <= k256 && tiles <= clusters) {
                p.splits = s;
                break;
            }
        }
        const int nA = (int)cdiv(k256, p.splits);
        p.own_digits = own;
        p.tmem_cols = small ? 256 : 512;
        p.smem = small ? kSmallSmem : kMaxSmem;
        const int room = p.smem - 1024 - (own ? nA * digits : 0), stage = stage_w + (own ? 0 : digits);
        p.stages_a = room < 0 ? 0 : imin(imin(kRowsStages, room / stage), (p.tmem_cols - p.d_cols - (int)cdiv(p.n_rows, 16) * 16 - 8) / 16);
        if (!own || (p.stages_a >= imin(small ? 4 : 6, nA + low) && nA <= kOwnTurns * own_warps(p.rows))) break;
    }
    return cudaSuccess;
}

cudaError_t launch_rows_fp4(const CUtensorMap& tm_w, const CUtensorMap& tm_s, const CUtensorMap& tm_x, const CUtensorMap& tm_l2,
                            const CUtensorMap& tm_u, const RowsParams& p, cudaStream_t st) {
    cudaError_t e = launch_rows_prepare(p, true, st);
    if (e != cudaSuccess) return e;
    if ((e = set_attributes()) != cudaSuccess) return e;
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
    return cudaLaunchKernelEx(&cfg, k_rows_fp4, tm_w, tm_s, tm_x, tm_l2, tm_u, p);
}

}  // namespace dq
