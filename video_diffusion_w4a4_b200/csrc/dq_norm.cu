// Root-mean-square norm of rows with the residual's addition (dq_rmsnorm_forward).
//
//   h = x + residual (fp32), sum = BF16(h),
//   y = h / sqrt(mean h^2 + eps) * gamma, stored as BF16 or as E4M3 codes with
//   s = max |y| / 448 per row or per 64 channels (the kernel tokens' rule).
//
// Bound by HBM: a row is read once into registers (pieces of eight channels, up
// to kMaxItems a thread), its sum of squares and maxima are formed there, and
// everything is written from there.  A row takes one CTA, or one warp when it
// has at most 1024 channels, so that narrow rows need no block-wide step.
// Eight neighbouring lanes hold 64 channels, so a group's maximum is three
// shuffles.  Pointers, strides and widths that do not allow 16-byte pieces take
// element accesses, for which a thread's channels are four pairs, a step of the
// row's threads apart: a warp's access is 128 bytes in a row then, and a step of a
// warp the 64 channels of a group.
//
// Measured on B200, residual added and stored, calls one after another:
// 32760 x 5120 to BF16 200 us (6.7 TB/s, the rate of a plain copy), 1560 x 5120 to
// E4M3 with group scales 13.9 us (4.0 TB/s; its bytes alone 8.6 us, the rest the
// launch, programmatic, 16.4 us without, and the last rows of 2.1 waves of CTAs).
// Rows of 257 to 1024 pieces take two a thread in CTAs of at most 512 threads,
// three or more to an SM: one piece a thread takes 16.9 us and 260 us, four CTAs'
// worth of registers (32) 14.9 and 222 us, gamma loaded before the sum 14.1 and 224 us.
// Element accesses: 1560 x 5119 to BF16 24 us, to E4M3 32 us per row and 35 us per group, 32760 x 1337 to
// BF16 110 us (46, 38, 35 and 228 us with eight neighbouring channels a thread).
#include <math.h>

#include "dq_common.h"
#include "dq_internal.h"
#include "dq_ptx.cuh"

namespace dq {

namespace {

constexpr int kMaxItems = 4;        // pieces of eight channels per thread
constexpr int kWarpRows = 4;        // rows per CTA when a row takes one warp

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Reduction over the threads of a row: a warp, or the whole CTA (every thread gets the result; each
// call uses its own 32 words of `sh`).
template <bool kWarp, typename T, typename Op>
__device__ __forceinline__ T row_reduce(T v, T* sh, Op op) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (!kWarp) {
        const int nw = (int)(blockDim.x >> 5), lane = threadIdx.x & 31;
        if (lane == 0) sh[threadIdx.x >> 5] = v;
        __syncthreads();
        T r = sh[0];
        for (int w = 1; w < nw; w++) r = op(r, sh[w]);
        v = r;
    }
    return v;
}

// Channel of thread t's value j (even; j + 1 has the next) in piece i of a row that T threads share
template <bool kWide>
__device__ __forceinline__ int channel(int t, int T, int i, int j) {
    return kWide ? 8 * (t + i * T) + j : 2 * (t + (4 * i + j / 2) * T);
}

// Piece i of a row (zeros past its end); BF16 bits, the low half of a word first.
template <bool kWide>
__device__ __forceinline__ void load8(const uint16_t* src, int t, int T, int i, int C, uint32_t (&w)[4]) {
    if (kWide) {
        const uint4 v = *reinterpret_cast<const uint4*>(src + channel<true>(t, T, i, 0));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int c = channel<false>(t, T, i, 2 * k);
            const uint32_t lo = c < C ? src[c] : 0, hi = c + 1 < C ? src[c + 1] : 0;
            w[k] = lo | (hi << 16);
        }
    }
}

template <bool kWide>
__device__ __forceinline__ void store8(uint16_t* dst, int t, int T, int i, int C, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; k++) w[k] = bf16x2_rn(v[2 * k], v[2 * k + 1]);
    if (kWide) {
        *reinterpret_cast<uint4*>(dst + channel<true>(t, T, i, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int c = channel<false>(t, T, i, 2 * k);
            if (c < C) dst[c] = (uint16_t)w[k];
            if (c + 1 < C) dst[c + 1] = (uint16_t)(w[k] >> 16);
        }
    }
}

// E4M3 codes of kPairs pairs y / s, two pairs a word, correctly rounded quotients; 0 where s is 0.
template <int kPairs>
__device__ __forceinline__ void codes(const float* y, float s, uint32_t* w) {
#pragma unroll
    for (int k = 0; k < (kPairs + 1) / 2; k++) w[k] = 0;
    if (s > 1e-30f && s < 1e30f) {
        const float rs = __frcp_rn(s);
#pragma unroll
        for (int k = 0; k < kPairs; k++) w[k / 2] |= cvt_e4m3x2(div_pos(y[2 * k], s, rs), div_pos(y[2 * k + 1], s, rs)) << (16 * (k & 1));
    } else if (s != 0.f) {
#pragma unroll
        for (int k = 0; k < kPairs; k++) w[k / 2] |= cvt_e4m3x2(__fdiv_rn(y[2 * k], s), __fdiv_rn(y[2 * k + 1], s)) << (16 * (k & 1));
    }
}

// The codes of a piece, two pairs a word
template <bool kWide>
__device__ __forceinline__ void store_codes8(uint8_t* dst, int t, int T, int i, int C, const uint32_t (&w)[2]) {
    if (kWide) {
        *reinterpret_cast<uint2*>(dst + channel<true>(t, T, i, 0)) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int c = channel<false>(t, T, i, 2 * k);
            const uint32_t two = w[k / 2] >> (16 * (k & 1));
            if (c < C) dst[c] = (uint8_t)two;
            if (c + 1 < C) dst[c + 1] = (uint8_t)(two >> 8);
        }
    }
}

enum { kOutBf16 = 0, kOutRow = 1, kOutGroup = 2 };

template <int kItems, bool kWarp, bool kWide, int kOut>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpRows : kItems == 2 ? 512 : 1024, kItems == 2 && !kWarp ? 3 : 1) k_rmsnorm(NormParams p) {
    __shared__ float sh[2][32];
    __shared__ double shd[32];
    const int T = kWarp ? 32 : (int)blockDim.x, t = kWarp ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    const long long row = kWarp ? (long long)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : (long long)blockIdx.x;
    if (kWarp && row >= p.rows) return;
    const uint16_t* x = p.x + row * p.x_stride;
    const uint16_t* r = p.residual + row * p.r_stride;
    griddep_wait();     // X may come from the launch before this one
    griddep_launch();
    uint32_t xw[kItems][4], rw[kItems][4];
#pragma unroll
    for (int i = 0; i < kItems; i++) {
        if (!kWide || channel<true>(t, T, i, 0) < p.C) {
            load8<kWide>(x, t, T, i, p.C, xw[i]);
            if (p.residual) load8<kWide>(r, t, T, i, p.C, rw[i]);
        }
    }
    float h[kItems][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < kItems; i++) {
#pragma unroll
        for (int j = 0; j < 8; j++) h[i][j] = 0.f;
        if (kWide && channel<true>(t, T, i, 0) >= p.C) continue;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            h[i][2 * j] = bf16_lo(xw[i][j]), h[i][2 * j + 1] = bf16_hi(xw[i][j]);
            if (p.residual) h[i][2 * j] += bf16_lo(rw[i][j]), h[i][2 * j + 1] += bf16_hi(rw[i][j]);
        }
#pragma unroll
        for (int j = 0; j < 8; j++) ss = fmaf(h[i][j], h[i][j], ss);
        if (p.sum) store8<kWide>(p.sum + row * p.s_stride, t, T, i, p.C, h[i]);
    }
    ss = row_reduce<kWarp>(ss, sh[0], [](float a, float b) { return a + b; });
    const float v = ss / (float)p.C + p.eps;
    float inv = rsqrtf(v);
    if (!(v > 0x1p-100f && v < 0x1p100f)) {
        // squares beyond fp32's range (or not finite): the same formula in 64 bits
        double sd = 0.0;
#pragma unroll
        for (int i = 0; i < kItems; i++)
#pragma unroll
            for (int j = 0; j < 8; j++) sd += (double)h[i][j] * h[i][j];
        sd = row_reduce<kWarp>(sd, shd, [](double a, double b) { return a + b; });
        const double id = 1.0 / sqrt(sd / p.C + (double)p.eps);
#pragma unroll
        for (int i = 0; i < kItems; i++)
#pragma unroll
            for (int j = 0; j < 8; j++) h[i][j] = (float)(h[i][j] * id);
        inv = 1.f;
    }
    float am = 0.f;
#pragma unroll
    for (int i = 0; i < kItems; i++) {
        const bool in = !kWide || channel<true>(t, T, i, 0) < p.C;   // (pairs are looked at one by one)
        if (in) {
            uint32_t gw[4];
            if (p.gamma) load8<kWide>(p.gamma, t, T, i, p.C, gw);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                h[i][j] *= inv;
                if (p.gamma) h[i][j] *= (j & 1) ? bf16_hi(gw[j / 2]) : bf16_lo(gw[j / 2]);
                // channels past the row's end take no part in a maximum (0 times infinity)
                if (!kWide && channel<false>(t, T, i, j & ~1) + (j & 1) >= p.C) h[i][j] = 0.f;
            }
        }
        if (kOut == kOutBf16) {
            if (in) store8<kWide>((uint16_t*)p.y + row * p.y_stride, t, T, i, p.C, h[i]);
        } else if (kOut == kOutRow) {
#pragma unroll
            for (int j = 0; j < 8; j++) am = max_nan(am, fabsf(h[i][j]));
        } else {
            uint32_t w[2] = {0, 0};
            float* scales = p.scales + row * ((p.C + 63) / 64);
            if (kWide) {
                // 64 channels sit in eight neighbouring lanes
                float a = fabsf(h[i][0]);
#pragma unroll
                for (int j = 1; j < 8; j++) a = max_nan(a, fabsf(h[i][j]));
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
                const float s = a / 448.0f;
                if (in) {
                    codes<4>(h[i], s, w);
                    store_codes8<true>((uint8_t*)p.y + row * p.y_stride, t, T, i, p.C, w);
                    if ((t & 7) == 0) scales[channel<true>(t, T, i, 0) / 64] = s;
                }
            } else {
                // ... or in the pairs of a warp
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    float a = max_nan(fabsf(h[i][2 * k]), fabsf(h[i][2 * k + 1]));
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
                    const float s = a / 448.0f;
                    uint32_t two;
                    codes<1>(&h[i][2 * k], s, &two);
                    w[k / 2] |= (two & 0xFFFFu) << (16 * (k & 1));
                    const int c = channel<false>(t, T, i, 2 * k);
                    if ((t & 31) == 0 && c < p.C) scales[c / 64] = s;
                }
                store_codes8<false>((uint8_t*)p.y + row * p.y_stride, t, T, i, p.C, w);
            }
        }
    }
    if (kOut == kOutRow) {
        const float s = row_reduce<kWarp>(am, sh[1], max_nan) / 448.0f;
#pragma unroll
        for (int i = 0; i < kItems; i++) {
            if (kWide && channel<true>(t, T, i, 0) >= p.C) continue;
            uint32_t w[2];
            codes<4>(h[i], s, w);
            store_codes8<kWide>((uint8_t*)p.y + row * p.y_stride, t, T, i, p.C, w);
        }
        if (t == 0) p.scales[row] = s;
    }
}

template <int kItems, bool kWarp, bool kWide>
cudaError_t launch(const NormParams& p, unsigned grid, unsigned threads, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (!p.scales) return cudaLaunchKernelEx(&cfg, k_rmsnorm<kItems, kWarp, kWide, kOutBf16>, p);
    if (!p.group) return cudaLaunchKernelEx(&cfg, k_rmsnorm<kItems, kWarp, kWide, kOutRow>, p);
    return cudaLaunchKernelEx(&cfg, k_rmsnorm<kItems, kWarp, kWide, kOutGroup>, p);
}

template <bool kWide>
cudaError_t launch_width(const NormParams& p, cudaStream_t st) {
    const int pieces = (int)cdiv(p.C, 8);
    const unsigned warp_grid = (unsigned)cdiv(p.rows, kWarpRows);
    if (pieces <= 32) return launch<1, true, kWide>(p, warp_grid, 32 * kWarpRows, st);
    if (pieces <= 64) return launch<2, true, kWide>(p, warp_grid, 32 * kWarpRows, st);
    if (pieces <= 128) return launch<4, true, kWide>(p, warp_grid, 32 * kWarpRows, st);
    const int items = pieces <= 256 ? 1 : pieces <= 1024 ? 2 : kMaxItems;
    const unsigned threads = (unsigned)(cdiv(cdiv(pieces, items), 32) * 32);
    if (items == 1) return launch<1, false, kWide>(p, (unsigned)p.rows, threads, st);
    if (items == 2) return launch<2, false, kWide>(p, (unsigned)p.rows, threads, st);
    return launch<kMaxItems, false, kWide>(p, (unsigned)p.rows, threads, st);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormParams& p, cudaStream_t st) {
    auto wide = [](const void* q, long long stride, int bytes) {
        return ((uintptr_t)q & (bytes - 1)) == 0 && stride * (bytes / 8) % bytes == 0;
    };
    // 16-byte pieces (8 bytes for codes) need every row of every buffer on that boundary
    const bool w = p.C % 8 == 0 && wide(p.x, p.x_stride, 16) && wide(p.residual, p.residual ? p.r_stride : 0, 16) &&
                   wide(p.gamma, 0, 16) && wide(p.sum, p.sum ? p.s_stride : 0, 16) &&
                   wide(p.y, p.y_stride, p.scales ? 8 : 16);
    return w ? launch_width<true>(p, st) : launch_width<false>(p, st);
}

}  // namespace dq
