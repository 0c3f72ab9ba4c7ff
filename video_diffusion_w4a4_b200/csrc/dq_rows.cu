// The product of few rows with a packed 4-bit weight (dq_rows_forward):
//   Y[m] = act( S_W sum_c xv[m][c] (q s_b)[o][c] + (xv[m] L1) L2 + b )
//
// With few rows the weight's bytes bound it: they cross from HBM once, and
// everything else hides behind that.  Two launches:
//
//   k_rows_prepare  rows -> the B operand, and U = xv L1.  FP16 holds every
//     q s_b exactly (6 significant bits, 2^-10 to 2688), so the product runs on
//     kind::f16 with FP16 operands, and a BF16 row is moved into FP16's range
//     by a power of two E of its own: x / E <= 2^15 keeps all 8 bits of values
//     down to 2^-29 of the row's largest, and is off by at most 2^-40 of the
//     largest below that, far under the fp32 sums' rounding.  E4M3 codes are
//     FP16 values already (E = the row's scale); with a scale per 64 channels
//     the row is code * scale, split into FP16 hi + lo (22 bits).  A cluster of
//     eight CTAs takes 16 rows, an eighth of the channels each, and joins its
//     maxima and its partial sums of U in a fixed order through distributed
//     shared memory; U / (E S_W) is kept as BF16 hi + lo, as in the cube layer.
//   k_rows_main     the product.  A CTA owns 128 output channels (the MMA's
//     rows) and up to 256 rows of X (its columns), and a part of the channels
//     when the tiles alone do not fill the GPU: the CTAs of a tile form a
//     cluster and sum their parts in rank order.  Codes and scales arrive by
//     TMA; eight warps turn them into FP16 (cvt.f16x2.e2m1x2, one product with
//     the group's scale) and put them into tensor memory, the MMA's A operand:
//     through shared memory they would cross it three times (write, and the
//     MMA's reads), which alone would take longer than the weight takes from
//     HBM.  The low-rank factor is extra BF16 K steps on the same accumulator.
//     The weight's loads do not wait for k_rows_prepare (programmatic launch).
#include "../../include/deltaquant.h"
#include "dq_common.h"
#include "dq_internal.h"
#include "dq_ptx.cuh"
#include "dq_rows.cuh"

namespace dq {

namespace {

// ------------------------------------------------------------------ PTX used by this file alone

__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// kind::f16, FP16 x FP16 -> fp32, K-major operands
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
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

// ------------------------------------------------------------------ the product

constexpr int kMainThreads = 384;               // producers (A, B), MMA, a spare warp, eight decoding warps
constexpr uint32_t kRowsStageA = kRowsCodeBytes + kRowsScaleBytes;   // 128 output x 256 input channels
constexpr int kMaxSmem = 225 * 1024;             // dynamic shared memory of a CTA that has an SM to itself

struct MainBars {
    uint64_t fullA[kRowsStages], emptyA[kRowsStages], fullB[kRowsStages], emptyB[kRowsStages], tfull[8], tempty[8], accf;
    uint32_t tmem;
    int abort_flag;
};

__global__ void __launch_bounds__(kMainThreads, 2)
    k_rows_main(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_s,
                const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_l2,
                const __grid_constant__ CUtensorMap tm_u, RowsParams p) {
    extern __shared__ __align__(16) uint8_t rows_smem[];
    uint8_t* sm = (uint8_t*)(((uintptr_t)rows_smem + 1023) & ~(uintptr_t)1023);
    __shared__ MainBars bars;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int SA = p.stages_a, SB = p.stages_b, R = p.ring;
    const uint32_t slotB = (uint32_t)p.n_pad * 128u;
    uint8_t* ringB = sm + (size_t)SA * kRowsStageA;
    volatile int* abort_flag = &bars.abort_flag;
    const int split = (int)blockIdx.x, splits = (int)gridDim.x;       // the cluster spans a tile's splits
    const int o0 = (int)blockIdx.y * 128;
    const int m0 = (int)blockIdx.z * p.n_rows;
    const int nm = imin(p.n_rows, p.rows - m0);
    const int k256 = p.Ci / 256, a0 = k256 * split / splits, nA = k256 * (split + 1) / splits - a0;
    const int chunks = 4 * nA, tiles = p.hilo ? 2 : 1;
    const int slabs = split == 0 ? p.slab / 64 : 0;

    if (tid == 0) {
        for (int s = 0; s < SA; s++) {
            mbar_init(&bars.fullA[s], 1);
            mbar_init(&bars.emptyA[s], 16);   // four chunks of a stage, four warps each
        }
        for (int s = 0; s < SB; s++) {
            mbar_init(&bars.fullB[s], 1);
            mbar_init(&bars.emptyB[s], 1);
        }
        for (int s = 0; s < R; s++) {
            mbar_init(&bars.tfull[s], 4);
            mbar_init(&bars.tempty[s], 1);
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
    const uint32_t tmem = bars.tmem, ring0 = tmem + (uint32_t)p.d_cols;

    if (warp == 0) {
        // ------------------------------------------------ codes and scales, then the low-rank factor's rows
        if (lane == 0) {
            const int total = nA + slabs, half = (o0 >> 7) & 1, blk0 = (o0 >> 8) * (p.Ci / 64) + a0 * 4;
            Ring r;
            int g = 0;
            for (; g < total; g++, r.next(SA)) {
                uint64_t* full = &bars.fullA[r.slot];
                if (g >= SA && !mbar_wait(&bars.emptyA[r.slot], r.phase ^ 1, abort_flag, p.status, p.budget_ns)) break;
                uint8_t* dst = sm + (size_t)r.slot * kRowsStageA;
                if (g < nA) {
                    mbar_arrive_expect_tx(full, kRowsStageA);
                    tma_load_2d(dst, &tm_w, full, (a0 + g) * 128, o0);
                    // 32 lanes x 16 bytes per 64-channel block: one half of the 256-row tile
                    tma_load_4d(dst + kRowsCodeBytes, &tm_s, full, 0, half, 0, blk0 + 4 * g);
                } else {
                    mbar_arrive_expect_tx(full, kRowsCodeBytes);
                    tma_load_2d(dst, &tm_l2, full, (g - nA) * 64, o0);
                }
            }
            for (int q = g > SA ? g - SA : 0; q < g; q++)   // every copy lands before shared memory is released
                mbar_wait(&bars.fullA[q % SA], (uint32_t)(q / SA) & 1, abort_flag, nullptr, p.budget_ns, false);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------ rows of X (FP16), then U
        if (lane == 0) {
            griddep_wait();
            const int main = chunks * tiles, total = main + slabs;
            int x = a0 * 256, low = 0;
            Ring r;
            int g = 0;
            for (; g < total; g++, r.next(SB)) {
                uint64_t* full = &bars.fullB[r.slot];
                if (g >= SB && !mbar_wait(&bars.emptyB[r.slot], r.phase ^ 1, abort_flag, p.status, p.budget_ns)) break;
                mbar_arrive_expect_tx(full, slotB);
                uint8_t* dst = ringB + (size_t)r.slot * slotB;
                if (g < main) {
                    tma_load_2d(dst, &tm_x, full, low + x, m0);
                    low = tiles == 2 && low == 0 ? p.Ci : 0;   // hi, then lo of the same channels
                    if (low == 0) x += 64;
                } else {
                    tma_load_2d(dst, &tm_u, full, (g - main) * 64, m0);
                }
            }
            for (int q = g > SB ? g - SB : 0; q < g; q++)
                mbar_wait(&bars.fullB[q % SB], (uint32_t)(q / SB) & 1, abort_flag, nullptr, p.budget_ns, false);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMAs (one elected lane; the warp's control flow is uniform)
        const uint32_t id_main = idesc_f16(128, p.n_pad), id_slab = idesc_bf16(128, p.n_pad);
        const uint64_t bdesc0 = desc_k_sw128(smem_u32(ringB));
        Ring rt, rb;
        bool alive = true;
        for (int c = 0; alive && c < chunks; c++, rt.next(R)) {
            if (!(alive = __all_sync(0xffffffffu, mbar_wait_spin(&bars.tfull[rt.slot], rt.phase, abort_flag, p.status, p.budget_ns)))) break;
            const uint32_t at = ring0 + (uint32_t)(32 * rt.slot);
            for (int h = 0; h < tiles; h++, rb.next(SB)) {
                if (!(alive = __all_sync(0xffffffffu, mbar_wait_spin(&bars.fullB[rb.slot], rb.phase, abort_flag, p.status, p.budget_ns)))) break;
                tc_fence_after();
                const uint64_t bd = bdesc0 + (uint64_t)((uint32_t)rb.slot * (slotB >> 4));
                if (elect_one()) {
                    mma_f16_ts(tmem, at, bd, id_main, (c | h) != 0);
                    mma_f16_ts(tmem, at + 8, bd + 2, id_main, 1u);
                    mma_f16_ts(tmem, at + 16, bd + 4, id_main, 1u);
                    mma_f16_ts(tmem, at + 24, bd + 6, id_main, 1u);
                    tc_commit(&bars.emptyB[rb.slot]);
                    if (h + 1 == tiles) tc_commit(&bars.tempty[rt.slot]);
                }
                __syncwarp();
            }
        }
        for (int i = 0; alive && i < slabs; i++, rb.next(SB)) {
            const int ga = nA + i, sa = ga % SA;
            if (!warp_wait(&bars.fullA[sa], (uint32_t)(ga / SA) & 1, abort_flag, p.status, p.budget_ns)) break;
            if (!warp_wait(&bars.fullB[rb.slot], rb.phase, abort_flag, p.status, p.budget_ns)) break;
            tc_fence_after();
            const uint64_t ad = desc_k_sw128(smem_u32(sm + (size_t)sa * kRowsStageA));
            const uint64_t bd = bdesc0 + (uint64_t)((uint32_t)rb.slot * (slotB >> 4));
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; k++) mma_bf16(tmem, ad + 2 * k, bd + 2 * k, id_slab, 1u);
                tc_commit(&bars.emptyB[rb.slot]);
            }
            __syncwarp();
        }
        if (elect_one()) {
            tc_commit(&bars.accf);
            mbar_wait(&bars.accf, 0, abort_flag, nullptr, p.budget_ns, false);   // no MMA runs past this point
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------ codes -> FP16 in tensor memory
        const int quad = warp & 3, group = (warp - 4) >> 2;   // 32 output channels; every other 64-channel chunk
        const int row = quad * 32 + lane;
        const uint32_t trow = ring0 + ((uint32_t)(quad * 32) << 16);
        // the TMA's 128-byte swizzle: 16-byte piece j of row r sits at piece j ^ (r % 8)
        const uint32_t at = (uint32_t)row * 128, x16 = (uint32_t)(row & 7);
        Ring ra, rt;
        rt.slot = group;   // the ring's size is even: a group keeps to its places
        for (int c = group; c < chunks; c += 2) {
            if (!warp_wait(&bars.fullA[ra.slot], ra.phase, abort_flag, p.status, p.budget_ns)) break;
            const uint8_t* st = sm + (size_t)ra.slot * kRowsStageA;
            const uint32_t j0 = 2 * (c & 3);
            const uint4 w0 = *reinterpret_cast<const uint4*>(st + at + ((j0 ^ x16) << 4));
            const uint4 w1 = *reinterpret_cast<const uint4*>(st + at + (((j0 + 1) ^ x16) << 4));
            const uint32_t sw = *reinterpret_cast<const uint32_t*>(st + kRowsCodeBytes + (c & 3) * 512 + lane * 16 + quad * 4);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.emptyA[ra.slot]);
            const uint32_t s01 = e4m3x2_to_f16x2(sw), s23 = e4m3x2_to_f16x2(sw >> 16);
            const uint32_t s0 = __byte_perm(s01, 0, 0x1010), s1 = __byte_perm(s01, 0, 0x3232);
            const uint32_t s2 = __byte_perm(s23, 0, 0x1010), s3 = __byte_perm(s23, 0, 0x3232);
            uint32_t v[16];
            decode8(w0.x, s0, v), decode8(w0.y, s0, v + 4), decode8(w0.z, s1, v + 8), decode8(w0.w, s1, v + 12);
            if (c >= R && !warp_wait(&bars.tempty[rt.slot], rt.phase ^ 1, abort_flag, p.status, p.budget_ns)) break;
            tc_fence_after();
            tmem_st_x16(trow + (uint32_t)(32 * rt.slot), v);
            uint32_t u[16];
            decode8(w1.x, s2, u), decode8(w1.y, s2, u + 4), decode8(w1.z, s3, u + 8), decode8(w1.w, s3, u + 12);
            tmem_st_x16(trow + (uint32_t)(32 * rt.slot + 16), u);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.tfull[rt.slot]);
            if ((c & 3) >= 2) ra.next(SA);
            rt.slot += 2;
            if (rt.slot >= R) rt.slot = group, rt.phase ^= 1;
        }
        __syncwarp();
    }

    // ---------------------------------------------------- epilogue
    const bool ok = header_ok(p);
    const PackedHeader* hdr = reinterpret_cast<const PackedHeader*>(p.packed_w);
    const float S_W = hdr->S_W;
    const float* bias = (hdr->flags & kPackedHasBias) ? (const float*)(p.packed_w + p.off_bias) : nullptr;
    bool done = true;
    if (warp >= 4) {
        done = warp_wait(&bars.accf, 0, abort_flag, p.status, p.budget_ns);
        tc_fence_after();
        griddep_wait();   // the rows' factors come from k_rows_prepare
    }
    const int quad = warp & 3, group = (warp - 4) >> 2, row = quad * 32 + lane;
    // Y of one output channel and the rows m, m + 1 (the second where it exists)
    auto finish = [&](int m, int o, float a0v, float a1v, float bv) {
        const float e0 = p.e[m0 + m], e1 = m + 1 < nm ? p.e[m0 + m + 1] : 0.f;
        float y0 = fmaf(a0v * S_W, e0, bv), y1 = fmaf(a1v * S_W, e1, bv);
        if (p.gelu) f2_unpack(gelu_erf2(f2_pack(y0, y1)), y0, y1);
        uint16_t* dst = p.y + (long long)(m0 + m) * p.y_stride + o;
        dst[0] = f32_to_bf16_rn(y0);
        if (m + 1 < nm) dst[p.y_stride] = f32_to_bf16_rn(y1);
    };
    if (splits == 1) {
        if (warp >= 4 && done && ok) {
            const float bv = bias ? bias[o0 + row] : 0.f;
            for (int c = 16 * group; c < nm; c += 32) {
                uint32_t acc[16];
                tmem_ld_x16(tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)c, acc);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; j += 2)
                    if (c + j < nm) finish(c + j, o0 + row, __uint_as_float(acc[j]), __uint_as_float(acc[j + 1]), bv);
            }
        }
    } else {
        // The parts of a tile: CTA r of the cluster sums, in rank order, the row pairs j with j % splits = r.
        // The buffer takes the operand ring's place, so every CTA of the cluster is past its MMAs first.
        __syncwarp();
        cluster_sync();
        float2* red = (float2*)sm;   // [source CTA][row pair / splits][128 output channels]
        const int pairs = (nm + 1) / 2, own = (pairs + splits - 1) / splits;
        if (warp >= 4 && done) {
            for (int c = 16 * group; c < nm; c += 32) {
                uint32_t acc[16];
                tmem_ld_x16(tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)c, acc);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const int pr = c / 2 + j;
                    if (pr < pairs) {
                        const uint32_t at = mapa_shared(smem_u32(&red[(split * own + pr / splits) * 128 + row]), pr % splits);
                        st_dsmem_f32(at, __uint_as_float(acc[2 * j]));
                        st_dsmem_f32(at + 4, __uint_as_float(acc[2 * j + 1]));
                    }
                }
            }
        }
        __syncwarp();
        cluster_sync();
        if (warp >= 4 && done && ok) {
            const int r = (tid - 128) & 127;
            const float bv = bias ? bias[o0 + r] : 0.f;
            for (int i = (tid - 128) >> 7; i * splits + split < pairs; i += 2) {
                float a = 0.f, b = 0.f;
                for (int q = 0; q < splits; q++) {
                    const float2 v = red[(q * own + i) * 128 + r];
                    a += v.x, b += v.y;
                }
                finish(2 * (i * splits + split), o0 + r, a, b, bv);
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

// How the product of `rows` rows is cut (RowsParams' fields from n_rows on).
void rows_plan(RowsParams& p) {
    // up to 256 rows of X a pass, evened out
    const int passes = (int)cdiv(p.rows, 256);
    p.n_rows = (int)cdiv(p.rows, passes);
    p.n_pad = (int)cdiv(p.n_rows, 16) * 16;
    p.passes = (int)cdiv(p.rows, p.n_rows);
    const bool small = p.n_pad <= 64;   // two CTAs per SM: 256 tensor-memory columns and 113 KB each
    p.tmem_cols = small ? 256 : 512;
    p.d_cols = small ? 64 : 256;
    p.ring = small ? 6 : 8;
    const int slot = p.n_pad * 128, room = small ? 110 * 1024 : kMaxSmem - 1024;
    p.stages_b = small ? (p.n_pad <= 16 ? 8 : p.n_pad <= 32 ? 6 : 4) : (p.n_pad <= 128 ? 6 : 4);
    p.stages_a = imin(kRowsStages, (room - p.stages_b * slot) / (int)kRowsStageA);
    p.smem = p.stages_a * (int)kRowsStageA + p.stages_b * slot + 1024;
    // as many parts of the channels as still let every CTA be resident at once
    const int tiles = p.Co / 128 * p.passes, places = small ? 296 : 148;
    p.splits = 1;
    while (p.splits < 8 && tiles * p.splits * 2 <= places && p.splits * 2 <= p.Ci / 256) p.splits *= 2;
}

cudaError_t launch_rows(const CUtensorMap& tm_w, const CUtensorMap& tm_s, const CUtensorMap& tm_x, const CUtensorMap& tm_l2,
                        const CUtensorMap& tm_u, const RowsParams& p, cudaStream_t st) {
    cudaError_t e = launch_rows_prepare(p, false, st);
    if (e != cudaSuccess) return e;
    e = once_per_device((const void*)k_rows_main, [] {
        return cudaFuncSetAttribute(k_rows_main, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
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
    return cudaLaunchKernelEx(&cfg, k_rows_main, tm_w, tm_s, tm_x, tm_l2, tm_u, p);
}

}  // namespace dq
