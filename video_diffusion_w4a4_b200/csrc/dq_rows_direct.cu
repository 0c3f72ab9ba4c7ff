// The product of up to 16 rows with a packed 4-bit weight (dq_rows_forward's
// smallest calls; dq_rows.cu has the mathematics and the form for more rows).
//
// So few rows leave nothing to hide latency behind but the weight's own loads,
// and a hand-off between producer, decoder and tensor memory costs more time
// per piece of weight than its HBM transfer.  Here a warp does everything for its
// piece: 32 output channels times 256 input channels at a time go from HBM into
// registers (32-byte loads, a full line per row and quad), are decoded to FP16
// there and are the A operand of mma.sync m16n8k16, eight rows of X its B
// operand.  The order of channels within an MMA's k is free as long as both
// operands use the same, so lane t of a quad owns channels 64 t to 64 t + 63 of
// the 256: its codes are one 32-byte load per output channel, its scales one
// 32-bit word, its values of X 128 consecutive bytes; nothing is exchanged or
// staged.  The 32 output channels are those whose scales share 16-byte pieces in
// the packed layout (32 c + i, c = 0..3, for eight i).  The warps of a CTA take
// the input channels in turns and add their sums through shared memory in a
// fixed order.
//
//   k_rows_lowrank   U = xv L1 in up to 16 partial sums over the channels
//   k_rows_direct    the product; its weight loads do not wait for U
//                    (programmatic launch), its epilogue adds U L2 and the bias.
//
// A BF16 row enters FP16 divided by a power of two 2^k that keeps its largest
// value so far in [2^14, 2^15); when a later step brings a larger one, the sums
// are scaled down to match (exact).  Values below 2^-29 of the largest lose bits,
// by at most 2^-40 of the largest (2^-25 for rows below 2^-112).  E4M3 codes are
// FP16 values; with a scale per 64 channels code * scale is split into hi + lo.
#include "../../include/deltaquant.h"
#include "dq_common.h"
#include "dq_internal.h"
#include "dq_ptx.cuh"
#include "dq_rows.cuh"

namespace dq {

namespace {

constexpr int kLowWarps = 8;

// Partial sums of U: CTA (chunk, 16 rows), each warp 64 channels at a time; lane t of a quad 16 of them.
template <int kNT, int kFmt>
__global__ void __launch_bounds__(32 * kLowWarps) k_rows_lowrank(RowsParams p) {
    extern __shared__ float low_sm[];   // [8 warps][16][rank]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int m0 = (int)blockIdx.y * 16, nm = imin(16, p.rows - m0), nblk = p.Ci / 64;
    const int b0 = nblk * (int)blockIdx.x / (int)gridDim.x, b1 = nblk * ((int)blockIdx.x + 1) / (int)gridDim.x;
    griddep_launch();
    float acc[kNT][4];
#pragma unroll
    for (int n = 0; n < kNT; n++)
#pragma unroll
        for (int i = 0; i < 4; i++) acc[n][i] = 0.f;
    for (int b = b0 + warp; b < b1; b += kLowWarps) {
        uint32_t xa[2][8];
        float sc[2];
        load_rows_16<kFmt>(p, m0, nm, b, g, t, xa, sc);
        lowrank_block<kNT, kFmt>(p, b, g, t, xa, sc, acc);
    }
    store_lowrank<kNT>(low_sm + warp * 16 * p.rank, p.rank, g, t, acc);
    __syncthreads();
    float* out = p.u_part + ((long long)blockIdx.x * p.rows + m0) * p.rank;
    for (int e = tid; e < nm * p.rank; e += 32 * kLowWarps) {
        float s = 0.f;
        for (int w = 0; w < kLowWarps; w++) s += low_sm[w * 16 * p.rank + e];
        out[e] = s;
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *p.status = header_ok(p) ? 0 : kStatusBadWeight;
}

struct Piece {           // a warp's 32 output channels x 256 input channels: this lane's codes and scales
    uint32_t w[4][8];
    uint32_t s[4];
};

__device__ __forceinline__ void ld_v8(const void* src, uint32_t (&v)[8]) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(src));
}

__device__ __forceinline__ void load_piece(const uint8_t* codes, size_t row32, const uint8_t* scales, int step, Piece& q) {
    const uint4 s = *reinterpret_cast<const uint4*>(scales + (size_t)step * 16384);
    q.s[0] = s.x, q.s[1] = s.y, q.s[2] = s.z, q.s[3] = s.w;
#pragma unroll
    for (int c = 0; c < 4; c++) ld_v8(codes + c * row32 + (size_t)step * 128, q.w[c]);
}

template <int kTiles, int kFmt>
__global__ void __launch_bounds__(512) k_rows_direct(RowsParams p) {
    extern __shared__ __align__(16) float direct_sm[];
    constexpr int kCols = 8 * kTiles, kPad = 36;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int W = (int)(blockDim.x >> 5), nm = p.rows;
    float* red = direct_sm;                                  // [W][kCols][36]
    float* su = red + W * kCols * kPad;                      // [rows][rank]
    uint32_t* l2s = (uint32_t*)(su + nm * p.rank);           // [32][rank / 2 + 1]
    const int rg = (int)blockIdx.x, tile = rg >> 3, half = (rg >> 2) & 1, i8 = rg & 3;
    const int obase = tile * 256 + half * 128 + i8 * 8;      // output channel of slot 8 c + i: obase + 32 c + i
    const int steps = p.Ci / 256, s0 = steps * warp / W, s1 = steps * (warp + 1) / W;
    const uint8_t* codes = p.packed_w + p.off_codes + (size_t)(obase + g) * (p.Ci / 2) + t * 32;
    const size_t row32 = (size_t)32 * (p.Ci / 2);
    const uint8_t* scales = p.packed_w + p.off_scales + ((size_t)tile * (p.Ci / 64) + t) * 4096 + i8 * 256 + half * 128 + g * 16;

    float acc[kTiles][2][4];
    int k[kTiles];
#pragma unroll
    for (int n = 0; n < kTiles; n++) {
        k[n] = -200;
#pragma unroll
        for (int i = 0; i < 8; i++) acc[n][i / 4][i % 4] = 0.f;
    }
    Piece cur, nxt;
    if (s0 < s1) load_piece(codes, row32, scales, s0, cur);
    // the low-rank factor's rows of these output channels
    for (int e = tid; e < 32 * (p.rank / 2); e += (int)blockDim.x) {
        const int slot = e / (p.rank / 2), j = e - slot * (p.rank / 2);
        l2s[slot * (p.rank / 2 + 1) + j] =
            *reinterpret_cast<const uint32_t*>(p.l2 + (size_t)(obase + 32 * (slot >> 3) + (slot & 7)) * p.slab + 2 * j);
    }
    for (int st = s0; st < s1; st++) {
        if (st + 1 < s1) load_piece(codes, row32, scales, st + 1, nxt);
        // this lane's 64 values of each row: raw, then FP16 pairs (hi, and lo with a scale per 64 channels)
        uint32_t xr[kTiles][kFmt == DQ_ROWS_BF16 ? 32 : 16];
        float gs[kTiles], inv[kTiles];
        bool grow = false;
#pragma unroll
        for (int n = 0; n < kTiles; n++) {
            const int m = 8 * n + g;
            constexpr int kWords = kFmt == DQ_ROWS_BF16 ? 32 : 16;
#pragma unroll
            for (int i = 0; i < kWords; i++) xr[n][i] = 0;
            gs[n] = 0.f;
            if (m < nm) {
                const char* src = (const char*)p.x + ((long long)m * p.x_stride + st * 256 + t * 64) * (kFmt == DQ_ROWS_BF16 ? 2 : 1);
#pragma unroll
                for (int i = 0; i < kWords; i += 4) {
                    const uint4 v = *reinterpret_cast<const uint4*>(src + 4 * i);
                    xr[n][i] = v.x, xr[n][i + 1] = v.y, xr[n][i + 2] = v.z, xr[n][i + 3] = v.w;
                }
                if (kFmt == DQ_ROWS_E4M3_GROUP64) gs[n] = p.x_scales[(long long)m * (p.Ci / 64) + st * 4 + t];
            }
            if (kFmt != DQ_ROWS_E4M3) {
                // the row's largest magnitude in these 256 channels, NaN above infinity above the rest
                float am;
                if (kFmt == DQ_ROWS_BF16) {
                    uint32_t a = 0;
#pragma unroll
                    for (int i = 0; i < kWords; i++) a = __vmaxu2(a, xr[n][i] & 0x7FFF7FFFu);
                    am = __uint_as_float((a & 0xFFFFu) > (a >> 16) ? a << 16 : a & 0xFFFF0000u);
                } else {
                    uint32_t a = 0;
#pragma unroll
                    for (int i = 0; i < kWords; i++) a = __vmaxu4(a, xr[n][i] & 0x7F7F7F7Fu);
                    a = max(max(a & 255u, (a >> 8) & 255u), max((a >> 16) & 255u, a >> 24));
                    am = fabsf(e4m3_to_f32(a) * gs[n]);
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
                const bool finite = am < __int_as_float(0x7F800000);
                int kn = !finite ? 999 : am > 0.f ? max(row_exponent(am), -126) : -200;
                kn = max(kn, k[n]);
                grow |= kn != k[n];
                inv[n] = kn == 999 ? __int_as_float(0x7FC00000) : kn == -200 ? 1.f : pow2i(-kn);
                if (__any_sync(0xffffffffu, kn != k[n])) {
                    // sums of the columns 2 t and 2 t + 1 move to the new power of two
                    const int d = k[n] - kn;
                    const float f = d < -126 ? 0.f : pow2i(d);
                    const float f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
                    for (int mt = 0; mt < 2; mt++) {
                        acc[n][mt][0] *= f0, acc[n][mt][1] *= f1;
                        acc[n][mt][2] *= f0, acc[n][mt][3] *= f1;
                    }
                    k[n] = kn;
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 4; q++) {   // 16 channels of the lane: one scale group
            uint32_t a[4][8];
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const uint32_t s = e4m3x2_to_f16x2(cur.s[c] >> (16 * (q >> 1)));
                const uint32_t ss = __byte_perm(s, 0, (q & 1) ? 0x3232 : 0x1010);
                decode8(cur.w[c][2 * q], ss, &a[c][0]);
                decode8(cur.w[c][2 * q + 1], ss, &a[c][4]);
            }
#pragma unroll
            for (int n = 0; n < kTiles; n++) {
#pragma unroll
                for (int i = 0; i < 4; i++) {   // MMA i of the group: channels 4 i to 4 i + 3 of every lane's 16
                    uint32_t b[2], lo[2];
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        if (kFmt == DQ_ROWS_BF16) {
                            const uint32_t r = xr[n][8 * q + 2 * i + e];
                            b[e] = f16x2_rn(bf16_lo(r) * inv[n], bf16_hi(r) * inv[n]);
                        } else {
                            const uint32_t h = e4m3x2_to_f16x2(xr[n][4 * q + i] >> (16 * e));
                            if (kFmt == DQ_ROWS_E4M3) {
                                b[e] = h;
                            } else {
                                float v0, v1, h0, h1;
                                f16x2_values(h, v0, v1);
                                v0 = v0 * gs[n] * inv[n], v1 = v1 * gs[n] * inv[n];
                                b[e] = f16x2_rn(v0, v1);
                                f16x2_values(b[e], h0, h1);
                                lo[e] = f16x2_rn(v0 - h0, v1 - h1);
                            }
                        }
                    }
#pragma unroll
                    for (int mt = 0; mt < 2; mt++) {
                        mma_16816_f16(acc[n][mt], a[2 * mt][2 * i], a[2 * mt + 1][2 * i], a[2 * mt][2 * i + 1],
                                      a[2 * mt + 1][2 * i + 1], b[0], b[1]);
                        if (kFmt == DQ_ROWS_E4M3_GROUP64)
                            mma_16816_f16(acc[n][mt], a[2 * mt][2 * i], a[2 * mt + 1][2 * i], a[2 * mt][2 * i + 1],
                                          a[2 * mt + 1][2 * i + 1], lo[0], lo[1]);
                    }
                }
            }
        }
        cur = nxt;
    }
    // S_W and the row's power of two, then the warps' sums in shared memory
    const PackedHeader* hdr = reinterpret_cast<const PackedHeader*>(p.packed_w);
    const float S_W = hdr->S_W;
#pragma unroll
    for (int n = 0; n < kTiles; n++) {
        float f0 = 1.f, f1 = 1.f;
        if (kFmt != DQ_ROWS_E4M3) {
            const float f = k[n] == 999 || k[n] == -200 ? 1.f : pow2i(k[n]);   // 999: the sums are NaN already
            f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
        }
        float* r0 = red + (warp * kCols + 8 * n + 2 * t) * kPad;
#pragma unroll
        for (int mt = 0; mt < 2; mt++) {
            r0[16 * mt + g] = acc[n][mt][0] * S_W * f0;
            r0[kPad + 16 * mt + g] = acc[n][mt][1] * S_W * f1;
            r0[16 * mt + 8 + g] = acc[n][mt][2] * S_W * f0;
            r0[kPad + 16 * mt + 8 + g] = acc[n][mt][3] * S_W * f1;
        }
    }
    griddep_wait();   // U
    for (int e = tid; e < nm * p.rank; e += (int)blockDim.x) {
        float s = 0.f;
        for (int c = 0; c < p.u_parts; c++) s += p.u_part[(long long)c * nm * p.rank + e];
        su[e] = s;
    }
    __syncthreads();
    if (!header_ok(p)) return;
    const float* bias = (hdr->flags & kPackedHasBias) ? (const float*)(p.packed_w + p.off_bias) : nullptr;
    const int slot = lane, o = obase + 32 * (slot >> 3) + (slot & 7);
    for (int m = warp; m < nm; m += W) {
        float y = 0.f, low = 0.f;
        for (int w = 0; w < W; w++) y += red[(w * kCols + m) * kPad + slot];
        for (int j = 0; j < p.rank / 2; j++) {
            const uint32_t l = l2s[slot * (p.rank / 2 + 1) + j];
            low = fmaf(su[m * p.rank + 2 * j], bf16_lo(l), low);
            low = fmaf(su[m * p.rank + 2 * j + 1], bf16_hi(l), low);
        }
        y += low;
        if (kFmt == DQ_ROWS_E4M3) y *= p.x_scales[m];
        if (bias) y += bias[o];
        if (p.gelu) {
            float unused;
            f2_unpack(gelu_erf2(f2_pack(y, 0.f)), y, unused);
        }
        p.y[(long long)m * p.y_stride + o] = f32_to_bf16_rn(y);
    }
}

template <int kNT>
cudaError_t launch_lowrank(const RowsParams& p, cudaStream_t st) {
    const size_t smem = (size_t)kLowWarps * 16 * p.rank * 4;
    const dim3 grid((unsigned)p.u_parts, (unsigned)cdiv(p.rows, 16));
    auto go = [&](auto kernel) {
        if (smem > 48 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
        }
        kernel<<<grid, 32 * kLowWarps, smem, st>>>(p);
        return cudaGetLastError();
    };
    if (p.x_format == DQ_ROWS_BF16) return go(k_rows_lowrank<kNT, DQ_ROWS_BF16>);
    if (p.x_format == DQ_ROWS_E4M3) return go(k_rows_lowrank<kNT, DQ_ROWS_E4M3>);
    return go(k_rows_lowrank<kNT, DQ_ROWS_E4M3_GROUP64>);
}

template <int kTiles, int kFmt>
cudaError_t launch_direct(const RowsParams& p, cudaStream_t st) {
    // warps per tile: all tiles' warps resident at once (16 per SM at this kernel's registers), 4 to 16
    const int tiles = p.Co / 32, steps = p.Ci / 256;
    int W = imin(16, (int)cdiv(16 * 148, tiles));
    W = imin(imin(W < 4 ? 4 : W, steps), 16);
    W = (int)cdiv(steps, cdiv(steps, W));
    const size_t smem = ((size_t)W * 8 * kTiles * 36 + (size_t)p.rows * p.rank + 32 * (p.rank / 2 + 1)) * 4;
    cudaError_t e = cudaSuccess;
    if (smem > 48 * 1024 && (e = cudaFuncSetAttribute(k_rows_direct<kTiles, kFmt>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                      (int)smem)) != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)tiles);
    cfg.blockDim = dim3((unsigned)(32 * W));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_rows_direct<kTiles, kFmt>, p);
}

}  // namespace

cudaError_t launch_rows_direct(const RowsParams& p, cudaStream_t st) {
    cudaError_t e = p.rank <= 16   ? launch_lowrank<2>(p, st)
                    : p.rank <= 32 ? launch_lowrank<4>(p, st)
                    : p.rank <= 64 ? launch_lowrank<8>(p, st)
                                   : launch_lowrank<16>(p, st);
    if (e != cudaSuccess) return e;
    if (p.rows <= 8) {
        if (p.x_format == DQ_ROWS_BF16) return launch_direct<1, DQ_ROWS_BF16>(p, st);
        if (p.x_format == DQ_ROWS_E4M3) return launch_direct<1, DQ_ROWS_E4M3>(p, st);
        return launch_direct<1, DQ_ROWS_E4M3_GROUP64>(p, st);
    }
    if (p.x_format == DQ_ROWS_BF16) return launch_direct<2, DQ_ROWS_BF16>(p, st);
    if (p.x_format == DQ_ROWS_E4M3) return launch_direct<2, DQ_ROWS_E4M3>(p, st);
    return launch_direct<2, DQ_ROWS_E4M3_GROUP64>(p, st);
}

}  // namespace dq
