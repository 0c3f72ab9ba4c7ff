// The product of few rows with a packed 4-bit weight (dq_rows_forward):
//   Y[m] = act( S_W sum_c xv[m][c] (q s_b)[o][c] + (xv[m] L1) L2 + b )
//
// Few rows leave the weight's bytes as the bound, and decoding codes costs more
// time than reading them.  Here they are not decoded: codes and group scales are
// the A operand of kind::mxf4nvf4 as they lie in the packed weight, and a row of X
// is written in the same format as kDigits = 8 FP4 digits a value,
//   x = 2^(e-1) sum_p 8^-p d_p + r,   d_p in {-4, ..., 4},  |r| <= 2^(e-23),
// with 2^e <= max |x| < 2^(e+1) over the row and d_p the nearest integer to what
// the digits before it leave: 24 bits below the row's largest value.  Each digit is a
// column of the MMA (the B scales are 1) and the epilogue sums a row's columns with
// their weights 8^-p in fp32.
//
// Digits hold a BF16 value whole from 2^(e-15) on, and E4M3 codes with one scale always.
// Smaller values lose bits, which an fp32 sum would keep where the weights of the larger
// ones are zero.  So a row of which more than an eighth of the values other than zero lie
// below 2^(e-15) is not taken from its digits: the epilogue forms its sums in fp32 from
// the values themselves (wide_rows; span_sum has the rule).  Rows of normally distributed
// values with outliers up to some 5000 times their deviation are on the digits' side.
//
// The low-rank factor is BF16 K steps of the same warp into columns of their own
// (U = xv L1 as hi + lo, times L2).
//
//   k_rows_product   128 output channels (the MMA's M) times up to 32 rows (256
//                    columns) per CTA.  One warp keeps codes and scales in flight,
//                    one the digits, one issues scale copies and MMAs, eight write
//                    the output.  When the tiles alone do not fill the GPU a cluster
//                    splits the channels and sums its parts in order through
//                    distributed shared memory.  From three passes over the rows
//                    on, CTA pairs (256 output channels, each CTA half of the digits'
//                    columns) take one piece of work after another.
//   k_rows_prepare   what it needs of the rows: digits and unit 2^(e-1), and U = xv
//                    L1, which the product multiplies with L2 as BF16 K steps (hi +
//                    lo) into columns of their own.
//
// With few rows k_rows_product does all of it (one launch): up to four where a CTA's
// digits and a ring of six stages fit, five to kOwnRows where it has four stages at most
// (rows_plan, own_turns).  The warps that write the output write the digits of the CTA's
// channels before it, and eight more form the low-rank term beside the product.  The CTAs of a cluster, parts of tiles
// and whole ones, take a share of the channels of U each and exchange their sums
// through distributed shared memory, so that L1 is read once a cluster.
//
// Bound: the weight's bytes (HBM) up to some 30 rows, then the digits: their MMAs and
// their traffic from L2 to the SMs, 4 bytes a value of X and tile of 128 output
// channels (2 with pairs).  Measured on B200, calls one after another on weights that
// are not in L2, against the time that the bytes of weight, factors, X and Y need at
// the HBM's copy rate:
//   1 x 5120 -> 5120     9.0 us (2.4)      1 x 5120 -> 13824   14.2 us (6.3)
//   4 x 13824 -> 5120   14.4 us (6.3)     21 x 5120 -> 13824   16.5 us (6.4)
//   77 x 2048 -> 5120   12.7 us (1.3)    512 x 5120 -> 5120    60 us (4.0; 16 at the
//   BF16 tensor rate)
// The stream alone, the same copies without any MMAs, takes 3.3 us for 5120 -> 5120
// and 7.1 us for 5120 -> 13824 (5.6 TB/s); a launch that waits for the one before it
// starts some 2.7 us after that one's last CTA has left (1.7 us until its wait
// returns, 1 us of setup), the first stage arrives 1.5 us later, and the output is
// written 1.3 to 1.9 us after the last MMA.  At 512 rows a pair's piece (5120 channels,
// 30 rows) takes 7.1 us, of which 5.3 us are MMAs at the tensor pipe's full rate and
// 1.8 us the accumulator's hand-over.
//
// MMAs: the four scale copies and four MMAs of a stage of 256 channels take 183
// cycles with 8 columns, 336 with 168 and 512 with 256 (the tensor pipe's full rate),
// issued by one lane without a pause.
//
// Once the weight streams, a load of anything else waits behind it for 2 to 4 us, a
// ring of the weight's stages per SM deep.  So the other loads come first, or where
// nothing waits for them: k_rows_product holds the stream back until they are under
// way (before the header's check: 5120 -> 5120 9.4 us against 9.8 us without, 5120 -> 13824
// 13.7 against 13.1, 13824 -> 5120 with 4 rows the same either way), and k_rows_prepare lets the product
// in when its own have arrived (programmatic launch).
#include "../../include/deltaquant.h"
#include "dq_common.h"
#include "dq_internal.h"
#include "dq_ptx.cuh"

#include <atomic>

namespace dq {

namespace {

constexpr int kDigits = 8;                       // FP4 digits of a value
constexpr int kPassRows = 32;                    // rows of X per CTA: 256 MMA columns
constexpr int kOwnRows = 8;                      // up to so many rows the product writes the digits itself
constexpr int kOwnTurns = 10;                    // pieces of eight channels a thread holds for that at most
// ... and uses: with a warp to a row (five rows and more) six and seven of them take longer than k_rows_prepare (8 rows:
// 4608 -> 5120 10.9 us against 10.5, 5120 -> 5120 11.5 against 10.5), four and fewer do not (2560 -> 5120 9.9 us against
// 10.1, 2048 -> 5120 9.3 against 10.7, 1280 -> 5120 9.0 against 10.8, 1536 -> 1536 7.8 against 10.1); five are as good
// either way (3840 -> 5120 10.2 against 10.7).  With two warps or more to a row ten take less (when measured, 4 rows,
// 5120 -> 13824: 14.2 us against 14.7 us; 13824 -> 5120: 16.0 us against 18.4 us).  A thread holds all of them in
// registers, whatever the row count: the E4M3 forms spill some 90 bytes of their 96 registers for it.
constexpr int own_turns(int rows) { return rows <= 4 ? kOwnTurns : 4; }
// producers of A and B, MMA, a spare warp, eight epilogue warps; eight for the low-rank term
constexpr int product_threads(bool own) { return own ? 640 : 384; }
constexpr int kEpiThreads = 256;
constexpr int kStages = 16;                      // stages of the operand ring at most
constexpr uint32_t kCodeBytes = 128 * 128;       // codes of 128 output channels x 256 input channels
constexpr uint32_t kScaleBytes = 4 * 512;        // their group scales
// Dynamic shared memory: a CTA has an SM to itself (so that none waits there for tensor memory while its cluster
// waits for it), and all of the tensor memory.
constexpr int kSmem = 224 * 1024;
constexpr uint32_t kTmemCols = 512;

// ------------------------------------------------------------------ small pieces

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void bar_arrive(int id, int nthreads) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// As mbar_wait, for a barrier that other CTAs of the cluster arrive on: acquires what they wrote before.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                                  uint64_t budget_ns) {
    const uint64_t t0 = globaltimer();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if (globaltimer() - t0 > budget_ns) {
            *abort_flag = 1;
            atomicCAS(status, 0, kStatusTimeout);
            return false;
        }
    }
}

// D(16 x 8) += A(16 x 16) B(16 x 8), BF16 operands, fp32 sums
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

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

// ... in both CTAs of a pair, each from its own shared memory to its own tensor memory
__device__ __forceinline__ void tmem_cp_pair_32x128b(uint32_t taddr, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

__device__ __forceinline__ void tma_load_4d_pair(void* dst, const CUtensorMap* map, uint32_t bar_cluster, int x, int y, int z,
                                                 int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(bar_cluster), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
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

// The two E2M1 codes of a byte -> FP16 pair (exact), the low nibble's in the low half
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t codes) {
    uint32_t h2;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.u8.u32 t, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
        : "=r"(h2)
        : "r"(codes));
    return h2;
}

// Two E4M3 codes -> FP16 pair (exact), the low byte's in the low half
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)codes));
    return h2;
}

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The packed weight's header up to its flags: magic, version, Co, Ci; rank, slab, S_W, flags.
struct Header {
    uint4 a, b;
};
__device__ __forceinline__ Header load_header(const RowsParams& p) {
    const uint4* h = reinterpret_cast<const uint4*>(p.packed_w);
    return Header{h[0], h[1]};
}

// ... ahead of the launches before this one, so that no L1 keeps it
__device__ __forceinline__ Header early_header(const RowsParams& p) {
    const uint4* h = reinterpret_cast<const uint4*>(p.packed_w);
    return Header{__ldcv(h), __ldcv(h + 1)};
}

// Nothing of a packed weight but its header may be read before this holds: its sections lie where this call's sizes
// say, and a weight of other sizes may end before them.  (The wait for it before the stream: 0.4 us of a call.)
__device__ __forceinline__ bool header_ok(const Header& h, const RowsParams& p) {
    return h.a.x == DQ_PACK_MAGIC && h.a.y == DQ_PACK_FORMAT_VERSION && (int)h.a.z == p.Co && (int)h.a.w == p.Ci &&
           (int)h.b.x == p.rank && (int)h.b.y == p.slab;
}

__device__ __forceinline__ void f16x2_values(uint32_t h2, float& lo, float& hi) {
    __half2_raw r;
    r.x = (uint16_t)(h2 & 0xFFFFu), r.y = (uint16_t)(h2 >> 16);
    const float2 f = __half22float2(__half2(r));
    lo = f.x, hi = f.y;
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

// ------------------------------------------------------------------ rows and digits

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

// Exponent of a row's unit, the weight of its first digit, from its largest magnitude: values stay below 4
// units; subnormals count as 2^-126.
__device__ __forceinline__ int unit_exponent(float am) {
    const int e = (int)((__float_as_uint(am) >> 23) & 255);
    return (e ? e - 127 : -126) - 1;
}

__device__ __forceinline__ bool finite_row(float am) { return am < __int_as_float(0x7F800000); }

// What a row's sum of digits is multiplied by: its unit 2^k, with the row's scale where the format has one; NaN
// for a row with a NaN or an infinity (in its values, whose digits are then zeros, or its scale).
template <int kFmt>
__device__ __forceinline__ float row_factor(const RowsParams& p, int m, int k, bool finite) {
    float E = k >= -126 ? pow2i(k) : __int_as_float(1 << (k + 149));
    if (kFmt == DQ_ROWS_E4M3) {
        const float s = p.x_scales[m];
        finite = finite && finite_row(fabsf(s));
        E *= s;
    }
    return finite ? E : __int_as_float(0x7FC00000);
}

// 2^-k in two exact steps (k in [-127, 126])
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

// A row's values v 2^-k count 7 where they are below 2^-14 (below 2^(e-15) of the row, where BF16 values lose
// bits as digits), -1 where they are not and nothing where they are zero: positive for a row of which more than
// an eighth is too small.  `v` and `raw` are the same eight values.
template <int kFmt>
__device__ __forceinline__ int span_sum(const Raw8<kFmt>& raw, const uint64_t (&v)[4], int k) {
    if (kFmt == DQ_ROWS_E4M3) return 0;   // exact in eight digits
    int sum = 0;
    if (kFmt == DQ_ROWS_BF16) {
        // by halves of a word: adding 2^15 less a bound sets a half's high bit from that bound on
        const int te = k + 1 - 15 + 127;
        const uint32_t small = (0x8000u - (te > 0 ? (uint32_t)te << 7 : 1u)) * 0x10001u;
        uint32_t large = 0, any = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t a = raw.w[i % (kFmt == DQ_ROWS_BF16 ? 4 : 2)] & 0x7FFF7FFFu;
            large |= ((a + small) & 0x80008000u) >> i;
            any |= ((a + 0x7FFF7FFFu) & 0x80008000u) >> i;
        }
        sum = 7 * __popc(any) - 8 * __popc(large);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float a, b;
            f2_unpack(v[i], a, b);
            sum += fabsf(a) >= 0x1p-14f ? -1 : a != 0.f ? 7 : 0;
            sum += fabsf(b) >= 0x1p-14f ? -1 : b != 0.f ? 7 : 0;
        }
    }
    return sum;
}

// Channels 64 b + 16 t to + 15 of the rows m0 + g and m0 + g + 8 (the second unless kHalf) as BF16 pairs (zeros from
// row nm on), and their scales where the format has one per 64 channels.
template <int kFmt, bool kHalf>
__device__ __forceinline__ void load_rows_16(const RowsParams& p, int m0, int nm, int b, int g, int t, uint32_t (&xa)[2][8],
                                             float (&sc)[2]) {
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int m = g + 8 * h;
#pragma unroll
        for (int i = 0; i < 8; i++) xa[h][i] = 0;
        sc[h] = 0.f;
        if ((kHalf && h) || m >= nm) continue;
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

// k_rows_prepare's CTAs: eight channels a thread, a row in as few of them as that allows.  Then a warp of a low-rank
// cluster has one 64-channel block, too.
// (77 rows of 2048: 12 us for the call, 14.8 us with 1024 threads whatever the row; 512 threads whatever the row
// cost 512 rows of 5120 7 us.)
constexpr int kPrepThreads = 1024, kPrepCluster = 8;
inline int prep_threads(int Ci) {
    const int warps = (int)cdiv(Ci, 256 * rows_parts(Ci));
    return 32 * (warps < 8 ? 8 : warps);
}

// Digits of the pieces (a row's channels that one CTA has at once) first, first + step, ... of all.  A CTA finds the
// row's largest magnitude for itself: a second read of at most 28 KB, from L2, costs less than a hand-off between
// CTAs.  The next piece's loads are under way beside this one's digits.
template <int kFmt>
__device__ __forceinline__ void digits_blocks(const RowsParams& p, int first, int step) {
    __shared__ float sh[2][kPrepThreads / 32];
    __shared__ int span[2];
    const int tid = threadIdx.x, lane = tid & 31, channels = 8 * (int)blockDim.x, parts = rows_parts(p.Ci), all = p.rows * parts;
    if (first >= all) return;
    if (tid < 2) span[tid] = 0;   // (the loop's barriers are between this and the sums)
    int last = -1;                // the piece before this one
    int m = parts == 1 ? first : first / parts, c = (first - m * parts) * channels + tid * 8;
    Raw8<kFmt> next = {};
    if (c < p.Ci) next = load_raw8<kFmt>(p, m, c);
    for (int at = first, turn = 0; at < all; turn ^= 1) {
        const Raw8<kFmt> raw = next;
        const int row = m, here = c;
        float am = amax8<kFmt>(raw);
        if (parts > 1)
            for (int i = tid * 8; i < p.Ci; i += channels)
                if (i != here) am = max_nan(am, amax8<kFmt>(load_raw8<kFmt>(p, row, i)));
        if ((at += step) < all) {
            m = parts == 1 ? at : at / parts, c = (at - m * parts) * channels + tid * 8;
            next = {};
            if (c < p.Ci) next = load_raw8<kFmt>(p, m, c);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
        if (lane == 0) sh[turn][tid >> 5] = am;
        __syncthreads();
        if (at >= all) griddep_launch();   // the CTA's loads have arrived
        // the piece before this one: its span is summed, as every thread is past that
        if (kFmt != DQ_ROWS_E4M3 && tid == 0 && last >= 0) p.span[last] = span[turn ^ 1], span[turn ^ 1] = 0;
        last = row * parts + (here - tid * 8) / channels;
        am = sh[turn][0];
        for (int w = 1; w < (int)blockDim.x / 32; w++) am = max_nan(am, sh[turn][w]);
        const bool finite = finite_row(am);
        const int k = unit_exponent(am);
        if (here == 0) p.e[row] = row_factor<kFmt>(p, row, k, finite);
        float v[8];
        uint64_t v2[4];
        values8<kFmt>(raw, v);
        scaled_pairs(v, inv_scale(k), finite, v2);
        if (kFmt != DQ_ROWS_E4M3) {
            const int s = __reduce_add_sync(0xffffffffu, finite ? span_sum<kFmt>(raw, v2, k) : 0);
            if (lane == 0) atomicAdd(&span[turn], s);
        }
        if (here >= p.Ci) continue;
        uint8_t* dst = p.digits + (size_t)row * kDigits * (p.Ci / 2) + here / 2;
#pragma unroll
        for (int q = 0; q < kDigits; q++) *reinterpret_cast<uint32_t*>(dst + (size_t)q * (p.Ci / 2)) = next_digits8(v2);
    }
    if (kFmt != DQ_ROWS_E4M3) {
        __syncthreads();
        if (tid == 0) p.span[last] = span[(all - 1 - first) / step & 1];
    }
}

// acc[n] += X L1 over the 64 channels of block b for 16 rows (or eight) and the ranks j0 + 8 n to + 7: lane t of a
// quad has 16 of the channels (any assignment of channels to the MMA's k is right that both operands share).  The
// loads are a call of their own, so that several blocks' can be under way.
template <bool kHalf>
struct LowRankBlock {
    uint32_t x[2][8];
    float s[2];
    uint4 l1[2][2];
};

template <int kFmt, bool kHalf>
__device__ __forceinline__ void lowrank_load(const RowsParams& p, int m0, int nm, int j0, int b, bool in, int g, int t,
                                             LowRankBlock<kHalf>& q) {
    load_rows_16<kFmt, kHalf>(p, m0, in ? nm : 0, b, g, t, q.x, q.s);
#pragma unroll
    for (int n = 0; n < 2; n++) {
        const uint4* src = reinterpret_cast<const uint4*>(p.l1 + (long long)(j0 + 8 * n + g) * p.Ci + b * 64 + t * 16);
        q.l1[n][0] = in ? src[0] : make_uint4(0, 0, 0, 0);
        q.l1[n][1] = in ? src[1] : make_uint4(0, 0, 0, 0);
    }
}

template <int kFmt, bool kHalf>
__device__ __forceinline__ void lowrank_add(const LowRankBlock<kHalf>& q, float (&acc)[2][4]) {
#pragma unroll
    for (int n = 0; n < 2; n++) {
        const uint4 u = q.l1[n][0], v = q.l1[n][1];
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma_16816(d, q.x[0][0], q.x[1][0], q.x[0][1], q.x[1][1], u.x, u.y);
        mma_16816(d, q.x[0][2], q.x[1][2], q.x[0][3], q.x[1][3], u.z, u.w);
        mma_16816(d, q.x[0][4], q.x[1][4], q.x[0][5], q.x[1][5], v.x, v.y);
        mma_16816(d, q.x[0][6], q.x[1][6], q.x[0][7], q.x[1][7], v.z, v.w);
        const float s0 = kFmt == DQ_ROWS_E4M3_GROUP64 ? q.s[0] : 1.f, s1 = kFmt == DQ_ROWS_E4M3_GROUP64 ? q.s[1] : 1.f;
        acc[n][0] = fmaf(d[0], s0, acc[n][0]);
        acc[n][1] = fmaf(d[1], s0, acc[n][1]);
        acc[n][2] = fmaf(d[2], s1, acc[n][2]);
        acc[n][3] = fmaf(d[3], s1, acc[n][3]);
    }
}

// Lane (g, t) holds the rows g and g + 8 and the ranks 8 n + 2 t and the next: into a row-major array of `rank` columns
template <bool kHalf>
__device__ __forceinline__ void lowrank_store(float* dst, int rank, int g, int t, const float (&acc)[2][4]) {
#pragma unroll
    for (int n = 0; n < 2; n++) {
        float* o = dst + g * rank + 8 * n + 2 * t;
        o[0] = acc[n][0], o[1] = acc[n][1];
        if (!kHalf) o[8 * rank] = acc[n][2], o[8 * rank + 1] = acc[n][3];
    }
}

// U of 16 rows and 32 ranks by a cluster of CTAs, a part of the channels each: a warp takes 16 of the ranks and one
// 64-channel block with eight CTAs (every so manieth with fewer, and past 8192 channels).  The sums are joined in rank order through distributed shared memory and
// kept as BF16 hi + lo, 2^-17 of the value.
template <int kFmt>
__device__ __forceinline__ void lowrank_cluster(const RowsParams& p, int index, float (*wpart)[16][32], float (*part)[32]) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int crank = (int)cluster_ctarank(), rgroups = (p.rank + 31) / 32;
    const int m0 = index / rgroups * 16, nm = imin(16, p.rows - m0), j0 = index % rgroups * 32;
    const int nblk = p.Ci / 64, csize = p.prep_cluster, sh = 31 - __clz(csize), b0 = nblk * crank >> sh, b1 = nblk * (crank + 1) >> sh;   // a power of two
    const int jw = j0 + 16 * (warp & 1), ks = warp >> 1, nks = (int)blockDim.x >> 6, warps = (int)blockDim.x >> 5;
    float acc[2][4] = {};
    if (jw < p.rank && ks < nks) {
        for (int b = b0 + ks; b < b1; b += nks) {
            LowRankBlock<false> q;
            lowrank_load<kFmt, false>(p, m0, nm, jw, b, true, g, t, q);
            lowrank_add<kFmt, false>(q, acc);
        }
    }
    if (ks < nks) lowrank_store<false>(&wpart[ks][0][16 * (warp & 1)], 32, g, t, acc);
    __syncthreads();
    griddep_launch();   // the CTA's loads have arrived
    for (int m = warp; m < 16; m += warps) {
        float u = 0.f;
        for (int k = 0; k < nks; k++) u += wpart[k][m][lane];
        part[m][lane] = u;
    }
    cluster_sync();
    // each CTA joins the sums of 16 / csize rows
    const int per = 16 >> sh;
    for (int i = warp; i < per; i += warps) {
        const int m = crank * per + i, j = j0 + lane;
        uint16_t* dst = p.u + (long long)(m0 + m) * p.slab;
        if (m < nm && j < p.rank) {
            const uint32_t at = smem_u32(&part[m][lane]);
            float v[kPrepCluster], u = 0.f;
#pragma unroll
            for (int c = 0; c < kPrepCluster; c++) v[c] = c < csize ? ld_dsmem_f32(mapa_shared(at, c)) : 0.f;
#pragma unroll
            for (int c = 0; c < kPrepCluster; c++) u += v[c];
            if (kFmt == DQ_ROWS_E4M3) u *= p.x_scales[m0 + m];
            const uint16_t hi = f32_to_bf16_rn(u);
            dst[j] = hi;
            dst[p.rank + j] = f32_to_bf16_rn(u - bf16_lo(hi));
        }
        // zeros up to the slab's width (at most 32 columns)
        if (m < nm && j0 == 0 && 2 * p.rank + lane < p.slab) dst[2 * p.rank + lane] = 0;
    }
    cluster_sync();   // no CTA leaves while another still reads its sums
}

template <int kFmt>
__global__ void __launch_bounds__(kPrepThreads) k_rows_prepare(RowsParams p) {
    griddep_wait();     // the launch before this one may still read the workspace, or write X
    __shared__ float wpart[16][16][32], part[16][32];
    // the low-rank clusters first: they take longest
    const int b = (int)blockIdx.x, low = (p.rows + 15) / 16 * ((p.rank + 31) / 32) * p.prep_cluster;
    if (b == 0 && threadIdx.x == 0) *p.status = header_ok(load_header(p), p) ? 0 : kStatusBadWeight;
    if (b < low)
        lowrank_cluster<kFmt>(p, b / p.prep_cluster, wpart, part);
    else
        digits_blocks<kFmt>(p, b - low, (int)gridDim.x - low);
}

// ------------------------------------------------------------------ the product

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

struct Bars {
    uint64_t full[kStages], empty[kStages], accf, acce, digits[kOwnTurns], u;
    float e[2][kPassRows];   // the rows' factors
    alignas(16) int span[2][kPassRows];  // positive: the row's values take the place of its digits
    alignas(16) float bias[128];
    float S_W;               // of the weight's header, with its flags, and whether it is this call's
    uint32_t flags;
    int fits;
    float amax[8];        // own digits: each warp's part of its row's largest magnitude
    uint32_t tmem;
    int abort_flag;
};

// The digits' scales: E4M3 1 in eight columns of the warp's lanes
__device__ __forceinline__ void ones(uint32_t taddr) {
    const uint32_t one = 0x38383838u;
    tmem_st_x4(taddr, one, one, one, one);
    tmem_st_x4(taddr + 4, one, one, one, one);
    tmem_st_wait();
}

// Own digits: the epilogue warps write the digits of this CTA's channels into shared memory as the MMA reads
// them, with the unit of the rows' values in these channels alone.  Each row takes own_warps(rows) warps, which
// hold all its values from one read and write the digits 256 channels a warp at a time, each such turn with a
// barrier of its own for the MMAs.
__host__ __device__ constexpr int own_warps(int rows) { return rows == 1 ? 8 : rows == 2 ? 4 : rows <= 4 ? 2 : 1; }

template <int kFmt>
__device__ __forceinline__ void load_own_rows(const RowsParams& p, int c0, int channels, Raw8<kFmt> (&raw)[kOwnTurns]) {
    const int ew = (int)(threadIdx.x >> 5) - 4, lane = threadIdx.x & 31;
    const int per = own_warps(p.rows), m = ew / per, part = ew % per, first = (part * 32 + lane) * 8;
#pragma unroll
    for (int i = 0; i < kOwnTurns; i++) {
        raw[i] = {};
        if (m < p.rows && first + i * per * 256 < channels) raw[i] = load_raw8<kFmt>(p, m, c0 + first + i * per * 256);
    }
}

template <int kFmt>
__device__ __forceinline__ void write_own_digits(const RowsParams& p, Bars& bars, uint8_t* dst, int channels,
                                                 const Raw8<kFmt> (&raw)[kOwnTurns]) {
    const int ew = (int)(threadIdx.x >> 5) - 4, lane = threadIdx.x & 31;
    const int per = own_warps(p.rows), m = ew / per, part = ew % per, first = (part * 32 + lane) * 8;
    float am = 0.f;
#pragma unroll
    for (int i = 0; i < kOwnTurns; i++) am = max_nan(am, amax8<kFmt>(raw[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
    if (lane == 0) bars.amax[ew] = am;
    bar_sync(1, kEpiThreads);
    for (int i = 0; i < per; i++) am = max_nan(am, bars.amax[m * per + i]);
    const bool finite = finite_row(am);
    const int k = unit_exponent(am);
    if (m < p.rows && part == 0 && lane == 0) bars.e[0][m] = row_factor<kFmt>(p, m, k, finite);
    const Scale2 s = inv_scale(k);
    int span = 0;
#pragma unroll
    for (int i = 0; i < kOwnTurns; i++) {
        const int c = first + i * per * 256;
        if (i * per * 256 < channels) {
            if (m < p.rows && c < channels) {
                float v[8];
                uint64_t v2[4];
                values8<kFmt>(raw[i], v);
                scaled_pairs(v, s, finite, v2);
                if (finite) span += span_sum<kFmt>(raw[i], v2, k);
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
    if (kFmt != DQ_ROWS_E4M3) {   // read behind the epilogue warps' next barrier
        span = __reduce_add_sync(0xffffffffu, span);
        if (m < p.rows && lane == 0) atomicAdd(&bars.span[0][m], span);
    }
}

// The sums sum_c (x_c 2^-k) (q s_b)[o + lane][c] over the channels 64 b0 to 64 b1 - 1 for the rows m to m + 3 (those
// below m + nm) and a warp's 32 output channels, from the values as they are: BF16 operands (weights q s_b, BF16 values and
// E4M3 codes are exact in BF16), fp32 sums, and the scale of a row's 64 channels on their sum.  `e` holds the rows' units
// 2^k.  Bound by the latency of its loads: 1 x 5120 -> 5120 takes 28 us with it, 512 x 5120 -> 5120 130 us where one
// row needs it and 1.7 ms where all do (the digits alone 8.7 and 59 us).  The next block's loads ahead of this one's
// products take a fifth off that, and cost the rows that do not need it 0.6 us in registers.
__device__ __forceinline__ float4 wide_rows(const uint8_t* codes, const uint8_t* scales, const void* x, long long x_stride,
                                         const float* x_scales, int Ci, int o, int m, int nm, int b0, int b1, const float* e) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float acc[2][4] = {}, inv[2];
#pragma unroll
    for (int i = 0; i < 2; i++) inv[i] = 2 * t + i < imin(nm, 4) ? __frcp_rn(e[2 * t + i]) : 0.f;
    const float inv_g = g < imin(nm, 4) ? __frcp_rn(e[g]) : 0.f;
    const __nv_bfloat162 unit = __float2bfloat162_rn(inv_g);
#pragma unroll 1
    for (int b = b0; b < b1; b++) {
        uint32_t xa[8] = {};
        float sc[2] = {1.f, 1.f};
        if (g < imin(nm, 4)) {
            const long long off = (long long)(m + g) * x_stride + b * 64 + t * 16;
            if (!x_scales) {
                const uint4* src = reinterpret_cast<const uint4*>((const uint16_t*)x + off);
                const uint4 u = src[0], v = src[1];
                const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const __nv_bfloat162 s = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), unit);
                    xa[i] = *reinterpret_cast<const uint32_t*>(&s);
                }
            } else {
                const uint4 u = *reinterpret_cast<const uint4*>((const uint8_t*)x + off);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 8; i++) xa[i] = e4m3x2_to_bf16x2(w[i / 2] >> (16 * (i & 1)));
            }
        }
        if (x_scales) {
#pragma unroll
            for (int i = 0; i < 2; i++)
                sc[i] = 2 * t + i < imin(nm, 4) ? x_scales[(long long)(m + 2 * t + i) * (Ci / 64) + b] * inv[i] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 2; j++) {
            uint32_t w[2][8];   // the channels 16 t to + 15 of the block, one group scale: any order of channels that both share
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int row = o + 16 * j + 8 * h + g;
                const uint2 q = *reinterpret_cast<const uint2*>(codes + (long long)row * (Ci / 2) + b * 32 + t * 8);
                const float s = e4m3_to_f32(scales[sfb_offset(row, 4 * b + t, Ci)]);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    float lo, hi;
                    f16x2_values(e2m1x2_to_f16x2((i < 4 ? q.x : q.y) >> (8 * (i & 3))), lo, hi);
                    w[h][i] = bf16x2_rn(lo * s, hi * s);
                }
            }
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 8; i += 2) mma_16816(d, w[0][i], w[1][i], w[0][i + 1], w[1][i + 1], xa[i], xa[i + 1]);
#pragma unroll
            for (int i = 0; i < 4; i++) acc[j][i] = fmaf(d[i], sc[i & 1], acc[j][i]);
        }
    }
    // lane (g, t) has the rows 2 t and 2 t + 1 of the channels g, g + 8, g + 16, g + 24: each lane takes its channel's
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int from = (lane & 7) * 4 + i / 2;
        const float a = __shfl_sync(0xffffffffu, acc[0][i & 1], from), b = __shfl_sync(0xffffffffu, acc[0][2 + (i & 1)], from);
        const float c = __shfl_sync(0xffffffffu, acc[1][i & 1], from), d = __shfl_sync(0xffffffffu, acc[1][2 + (i & 1)], from);
        v[i] = lane < 8 ? a : lane < 16 ? b : lane < 24 ? c : d;
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}

// As a call of its own it leaves the one-launch form its registers (5120 -> 5120 8.7 us, 8.8 us inline); in the others
// the call costs more than it spares (21 x 5120 -> 13824 16.5 us, 16.3 us inline; 512 x 5120 -> 5120 62.6 and 60.3 us).
__device__ __noinline__ float4 wide_rows_call(const uint8_t* codes, const uint8_t* scales, const void* x, long long x_stride,
                                              const float* x_scales, int Ci, int o, int m, int nm, int b0, int b1, const float* e) {
    return wide_rows(codes, scales, x, x_stride, x_scales, Ci, o, m, nm, b0, b1, e);
}

// Low-rank term beside the product (at most kOwnRows rows): this CTA's share of the channels of U, cut further among
// eight warps (16 ranks x every u_parts-th block of 64 channels), exchanged within the cluster, then U L2 for the
// rows that this CTA finishes: low[i][output channel] of row split + i splits.
template <int kFmt>
__device__ __forceinline__ void lowrank_term(const RowsParams& p, Bars& bars, float* up, float* su, float* low, int o0,
                                             int crank, int csize, int split, int splits) {
    const int ut = (int)threadIdx.x - 384, uw = ut >> 5, lane = ut & 31, g = lane >> 2, t = lane & 3;
    const int items = p.rank / 16, nblk = p.Ci / 64, b0 = nblk * crank / csize, b1 = nblk * (crank + 1) / csize;
    const int row = ut & 127, mine = split < p.rows ? (p.rows - split + splits - 1) / splits : 0;
    const uint4* l2 = reinterpret_cast<const uint4*>(p.l2 + (size_t)(o0 + row) * p.slab);
    uint4 l2w[4];   // the first 32 ranks of this thread's output channel
#pragma unroll
    for (int j = 0; j < 4; j++) l2w[j] = 8 * j < p.rank ? l2[j] : make_uint4(0, 0, 0, 0);
    bool first = true;
    for (int w = uw; w < items * p.u_parts; w += 8) {
        const int part = w / items, j0 = (w - part * items) * 16;
        float acc[2][4] = {};
        for (int b = b0 + part; first || b < b1; b += 2 * p.u_parts) {
            LowRankBlock<true> q[2];
#pragma unroll
            for (int h = 0; h < 2; h++) lowrank_load<kFmt, true>(p, 0, p.rows, j0, b + h * p.u_parts, b + h * p.u_parts < b1, g, t, q[h]);
            if (first) bar_arrive(3, 32 + 512);   // the weight may follow
            first = false;
#pragma unroll
            for (int h = 0; h < 2; h++) lowrank_add<kFmt, true>(q[h], acc);
        }
        lowrank_store<true>(up + part * 8 * p.rank + j0, p.rank, g, t, acc);
    }
    if (first) bar_arrive(3, 32 + 512);
    bar_sync(4, 256);
    for (int e = ut; e < 8 * p.rank; e += 256) {
        float s = up[e];
        for (int k = 1; k < p.u_parts; k++) s += up[k * 8 * p.rank + e];
        up[e] = s;
    }
    bar_sync(4, 256);
    cluster_wait();
    if (ut < csize) mbar_arrive_cluster(mapa_shared(smem_u32(&bars.u), (uint32_t)ut));
    mbar_wait_cluster(&bars.u, 0, &bars.abort_flag, p.status, p.budget_ns);
    for (int e = ut; e < p.rows * p.rank; e += 256) {
        const uint32_t at = smem_u32(&up[e]);
        float v[8], u = 0.f;
#pragma unroll
        for (int c = 0; c < 8; c++) v[c] = c < csize ? ld_dsmem_f32(mapa_shared(at, (uint32_t)c)) : 0.f;
#pragma unroll
        for (int c = 0; c < 8; c++) u += v[c];
        if (kFmt == DQ_ROWS_E4M3) u *= p.x_scales[e / p.rank];
        su[e] = u;
    }
    bar_sync(4, 256);
    for (int i = ut >> 7; i < mine; i += 2) {
        const float* u = su + (split + i * splits) * p.rank;
        float y = 0.f;
        for (int j0 = 0; j0 < p.rank; j0 += 32) {
            if (j0) {
#pragma unroll
                for (int j = 0; j < 4; j++) l2w[j] = j0 + 8 * j < p.rank ? l2[j0 / 8 + j] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (j0 + 8 * j >= p.rank) break;
                const float4 u0 = *reinterpret_cast<const float4*>(u + j0 + 8 * j), u1 = *reinterpret_cast<const float4*>(u + j0 + 8 * j + 4);
                y = fmaf(u0.x, bf16_lo(l2w[j].x), y), y = fmaf(u0.y, bf16_hi(l2w[j].x), y);
                y = fmaf(u0.z, bf16_lo(l2w[j].y), y), y = fmaf(u0.w, bf16_hi(l2w[j].y), y);
                y = fmaf(u1.x, bf16_lo(l2w[j].z), y), y = fmaf(u1.y, bf16_hi(l2w[j].z), y);
                y = fmaf(u1.z, bf16_lo(l2w[j].w), y), y = fmaf(u1.w, bf16_hi(l2w[j].w), y);
            }
        }
        low[i * 128 + row] = y;
        if (p.rank > 32 && i + 2 < mine) {
#pragma unroll
            for (int j = 0; j < 4; j++) l2w[j] = l2[j];
        }
    }
    bar_arrive(5, 512);   // the epilogue warps wait for it
}

// The product's forms: from prepared rows, from rows whose digits it writes itself, and from prepared rows by CTA pairs
// (two tiles of output channels, each CTA with half of the digits' columns in its shared memory).
enum { kPrepared = 0, kOwnDigits = 1, kPairs = 2 };

// Registers a thread: 80 for prepared rows and 96 (the one-launch form's 640 threads) otherwise, as wide_rows would take
// up to 168, with which k_rows_prepare's CTAs do not fit beside this kernel's (the same times within 1 %).
template <int kFmt, int kForm>
__global__ void __launch_bounds__(product_threads(kForm != kPrepared), kForm == kPrepared ? 2 : 1)
    k_rows_product(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_s,
                   const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_l2,
                   const __grid_constant__ CUtensorMap tm_u, RowsParams p) {
    extern __shared__ __align__(16) uint8_t rows_smem[];
    uint8_t* sm = (uint8_t*)(((uintptr_t)rows_smem + 1023) & ~(uintptr_t)1023);
    __shared__ Bars bars;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = p.stages;
    constexpr bool own = kForm == kOwnDigits, pairs = kForm == kPairs;
    const int split = pairs ? 0 : (int)blockIdx.x, splits = pairs ? 1 : (int)gridDim.x;   // parts of the channels
    const int csize = splits * p.group, crank = (int)cluster_ctarank();   // in the cluster: those of `group` tiles
    // a CTA's work: one tile of output channels and one pass over rows; pairs take one such piece after another
    const int tiles = p.Co / 256, item0 = pairs ? (int)blockIdx.y : 0, items = pairs ? tiles * p.passes : 1,
              step = pairs ? (int)gridDim.y : 1;
    auto tile_of = [&](int item) { return pairs ? (item % tiles * 2 + crank) * 128 : (int)blockIdx.y * 128; };
    auto rows_of = [&](int item) { return (pairs ? item / tiles : (int)blockIdx.z) * p.n_rows; };
    int o0 = tile_of(item0), m0 = rows_of(item0), nm = imin(p.n_rows, p.rows - m0);   // the epilogue's piece at hand
    const int k256 = p.Ci / 256, a0 = k256 * split / splits, nA = k256 * (split + 1) / splits - a0;
    const uint32_t b_all = (uint32_t)p.n_pad * (pairs ? 64u : 128u), b_bytes = own ? 0u : b_all;   // digits of a stage; those in the ring
    const uint32_t stage = kCodeBytes + b_bytes + kScaleBytes;        // codes, digits, the codes' scales
    uint8_t* digits = sm + (size_t)S * stage;                         // own digits: [stage][column][128 bytes]
    const int total = nA + (!own && split == 0 ? p.slab / 64 : 0);    // stages: the weight's, then the low-rank factor's
    float* up = (float*)(digits + (own ? (size_t)p.own_stages * b_all : 0));   // own: [u_parts][8][rank] parts of U,
    float* su = up + p.u_parts * 8 * p.rank;                          //   U, U L2
    float* slow = su + 8 * p.rank;
    const uint32_t n16 = (uint32_t)(p.n_rows + 15) & ~15u;
    volatile int* abort_flag = &bars.abort_flag;
    // The header, on its way beside the setup: it lets the weight's loads start.  What is written to Y and reported goes
    // by another look at it behind the launches before this one, which may only now be writing it.
    Header early = {};
    if (warp == 0) early = early_header(p);

    if (tid == 0) {
        for (int s = 0; s < S; s++) {
            mbar_init(&bars.full[s], own ? 1 : 2);   // one producer, or both
            mbar_init(&bars.empty[s], 1);
        }
        for (int i = 0; i < kOwnTurns; i++) mbar_init(&bars.digits[i], kEpiThreads / 32);
        mbar_init(&bars.u, (uint32_t)(csize + p.u_missing));
        mbar_init(&bars.accf, 1);
        mbar_init(&bars.acce, 2 * kEpiThreads / 32);
        bars.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        if (pairs) {
            tmem_alloc_pair(&bars.tmem, kTmemCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&bars.tmem, kTmemCols);
            tmem_relinquish();
        }
    }
    if (tid >= 128 && tid < 128 + 2 * kPassRows) (&bars.span[0][0])[tid - 128] = 0;   // also of rows that there are not
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tm_w);
        prefetch_tmap(&tm_s);
        if (!own) {
            prefetch_tmap(&tm_x);
            prefetch_tmap(&tm_l2);
            prefetch_tmap(&tm_u);
        }
    }
    tc_fence_before();
    __syncwarp();
    if (pairs)
        cluster_sync();   // both CTAs' barriers are initialised
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem, t_low = tmem + (uint32_t)p.d_cols, t_one = t_low + n16, t_sf = t_one + 8;
    if (own) {
        cluster_arrive();   // waited for before this CTA first touches another's shared memory
        griddep_wait();     // with k_rows_prepare in front everything before that launch is done already
    }
    griddep_launch();
    const bool lead = !pairs || crank == 0;   // the CTA that issues the MMAs, and has the stages' full barriers
    if (pairs) {
        if (warp >= 4 && warp < 8) ones(t_one + ((uint32_t)((warp & 3) * 32) << 16));
        tc_fence_before();
        __syncwarp();
        cluster_sync();
        tc_fence_after();
    }

    if (warp == 0) {
        // ------------------------------------------------ codes and their scales
        if (own) bar_sync(3, 32 + 512);   // the loads of everything else are under way
        if (lane == 0) {
            Ring r;
            int n = 0;   // stages so far
            bool ok = true;
            const bool good = header_ok(early, p) || header_ok(load_header(p), p);   // else the stages stay as they are, and so does Y
            for (int item = item0; item < items && ok; item += step) {
                const int o = tile_of(item), half = (o >> 7) & 1, blk0 = (o >> 8) * (p.Ci / 64) + a0 * 4;
                for (int g = 0; g < total; g++, n++, r.next(S)) {
                    uint64_t* full = &bars.full[r.slot];
                    if (n >= S && !(ok = mbar_wait(&bars.empty[r.slot], r.phase ^ 1, abort_flag, p.status, p.budget_ns))) break;
                    uint8_t* dst = sm + (size_t)r.slot * stage;
                    if (!good) {
                        if (lead) mbar_arrive(full);
                    } else if (pairs) {
                        if (lead) mbar_arrive_expect_tx(full, 2 * (g < nA ? kCodeBytes + kScaleBytes : kCodeBytes));
                        const uint32_t at = mapa_shared(smem_u32(full), 0);
                        if (g < nA) {
                            tma_load_2d_pair(dst, &tm_w, at, (a0 + g) * 128, o);
                            tma_load_4d_pair(dst + kCodeBytes + b_bytes, &tm_s, at, 0, half, 0, blk0 + 4 * g);
                        } else {
                            tma_load_2d_pair(dst, &tm_l2, at, (g - nA) * 64, o);
                        }
                    } else if (g < nA) {
                        mbar_arrive_expect_tx(full, kCodeBytes + kScaleBytes);
                        tma_load_2d(dst, &tm_w, full, (a0 + g) * 128, o);
                        // 32 lanes x 16 bytes per 64-channel block: one half of the 256-row tile
                        tma_load_4d(dst + kCodeBytes + b_bytes, &tm_s, full, 0, half, 0, blk0 + 4 * g);
                    } else {
                        mbar_arrive_expect_tx(full, kCodeBytes);
                        tma_load_2d(dst, &tm_l2, full, (g - nA) * 64, o);
                    }
                }
            }
            // every copy lands before shared memory is released (a pair's second CTA: the MMAs have read them)
            for (int q = n > S ? n - S : 0; q < n; q++)
                mbar_wait(lead ? &bars.full[q % S] : &bars.empty[q % S], (uint32_t)(q / S) & 1, abort_flag, nullptr, p.budget_ns, !lead);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------ digits, then U
        if (lane == 0 && !own) {
            griddep_wait();
            Ring r;
            int n = 0;
            bool ok = true;
            for (int item = item0; item < items && ok; item += step) {
                const int m = rows_of(item);
                for (int g = 0; g < total; g++, n++, r.next(S)) {
                    uint64_t* full = &bars.full[r.slot];
                    if (n >= S && !(ok = mbar_wait(&bars.empty[r.slot], r.phase ^ 1, abort_flag, p.status, p.budget_ns))) break;
                    uint8_t* dst = sm + (size_t)r.slot * stage + kCodeBytes;
                    if (lead) mbar_arrive_expect_tx(full, g < nA ? (pairs ? 2 : 1) * b_bytes : n16 * 128);   // U in the digits' place
                    if (pairs) {
                        const uint32_t at = mapa_shared(smem_u32(full), 0);
                        if (g < nA)
                            tma_load_2d_pair(dst, &tm_x, at, (a0 + g) * 128, m * kDigits + crank * (p.n_pad / 2));
                        else
                            tma_load_2d_pair(dst, &tm_u, at, (g - nA) * 64, m + crank * (int)(n16 / 2));
                    } else if (g < nA) {
                        tma_load_2d(dst, &tm_x, full, (a0 + g) * 128, m * kDigits);
                    } else {
                        tma_load_2d(dst, &tm_u, full, (g - nA) * 64, m);
                    }
                }
            }
            for (int q = n > S ? n - S : 0; q < n; q++)
                mbar_wait(lead ? &bars.full[q % S] : &bars.empty[q % S], (uint32_t)(q / S) & 1, abort_flag, nullptr, p.budget_ns, !lead);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMAs, by one lane throughout
        if (!pairs) bar_sync(2, 32 + 128);   // the digits' scales are in tensor memory
        tc_fence_after();
        if (lead && elect_one()) {
            constexpr int M = pairs ? 256 : 128;
            const uint32_t idesc = idesc_nvfp4(M, p.n_pad), id_low = idesc_bf16(M, (int)n16);
            // descriptors: the address field is the offset / 16, so a step is an addition
            const uint32_t base = smem_u32(sm), step16 = stage >> 4, b_step = own ? b_all >> 4 : step16;
            const uint64_t a0d = desc_k_sw128(base), b0d = desc_k_sw128(own ? smem_u32(digits) : base + kCodeBytes),
                           f0d = smem_desc(base + kCodeBytes + b_bytes, 128, 128, 0);
            auto commit = [](uint64_t* bar) {
                if (pairs)
                    tc_commit_pair_both(bar, 3);
                else
                    tc_commit(bar);
            };
            Ring r;
            uint64_t ad = a0d, bd = b0d, fd = f0d;
            uint32_t ta = t_sf, used = 0;                    // pieces so far
            int turn = 0, left = 0;                          // own digits: stages until the next turn's barrier
            const int per = own_warps(p.rows);
            bool ok = true;
            for (int item = item0; item < items && ok; item += step, used++) {
                if (used && !mbar_wait_spin(&bars.acce, (used - 1) & 1, abort_flag, p.status, p.budget_ns)) break;
                tc_fence_after();
                uint32_t more = 0;
                for (int g = 0; g < total; g++) {
                    if (own && left-- == 0) {
                        if (!(ok = mbar_wait_spin(&bars.digits[turn], 0, abort_flag, p.status, p.budget_ns))) break;
                        turn++;
                        left = per - 1;
                    }
                    if (!(ok = mbar_wait_spin(&bars.full[r.slot], r.phase, abort_flag, p.status, p.budget_ns))) break;
                    tc_fence_after();
                    if (own || g < nA) {
                        // the stage's own columns: nothing still reads them, as its empty barrier was waited for
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            if (pairs)
                                tmem_cp_pair_32x128b(ta + 4 * j, fd + 32 * j);
                            else
                                tmem_cp_32x128b(ta + 4 * j, fd + 32 * j);
                        }
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            if (pairs)
                                mma_nvfp4_pair(tmem, ad + 2 * j, bd + 2 * j, idesc, ta + 4 * j, t_one, j ? 1u : more);
                            else
                                mma_nvfp4(tmem, ad + 2 * j, bd + 2 * j, idesc, ta + 4 * j, t_one, j ? 1u : more);
                        }
                        more = g + 1 != nA;   // the low-rank factor's steps have columns of their own
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            if (pairs)
                                mma_bf16_pair(t_low, ad + 2 * j, bd + 2 * j, id_low, more | (uint32_t)j);
                            else
                                mma_bf16(t_low, ad + 2 * j, bd + 2 * j, id_low, more | (uint32_t)j);
                        }
                        more = 1;
                    }
                    commit(&bars.empty[r.slot]);
                    ad += step16, bd += b_step, fd += step16, ta += 16;
                    r.next(S);
                    if (r.slot == 0) {
                        ad = a0d, fd = f0d, ta = t_sf;
                        if (!own) bd = b0d;
                    }
                }
                if (!ok) {   // the accumulator is not whole: neither CTA's epilogue takes it when it arrives
                    *abort_flag = 1;
                    if (pairs) st_dsmem_f32(mapa_shared(smem_u32(&bars.abort_flag), 1), 1.f);
                    asm volatile("fence.acq_rel.cluster;" ::: "memory");
                }
                commit(&bars.accf);
            }
            if (used) mbar_wait(&bars.accf, (used - 1) & 1, abort_flag, nullptr, p.budget_ns, false);   // no MMA runs past this point
        }
        __syncwarp();
    }

    if (warp == 3) {
        // ------------------------------------------------ the header, S_W and the bias (the first piece's), for the epilogue
        const Header h = load_header(p);
        const bool fits = header_ok(h, p);
        float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
        if (fits && (h.b.w & kPackedHasBias)) b = *reinterpret_cast<const float4*>(p.packed_w + p.off_bias + 4ll * (o0 + 4 * lane));
        *reinterpret_cast<float4*>(&bars.bias[4 * lane]) = b;
        if (lane == 0) {
            bars.S_W = __uint_as_float(h.b.z);
            bars.flags = h.b.w;
            bars.fits = fits;
            // the call's status word, long before a wait of any CTA can have run out and been recorded there
            if (own && blockIdx.x + blockIdx.y + blockIdx.z == 0) *p.status = fits ? 0 : kStatusBadWeight;
        }
        __syncwarp();
        bar_arrive(6, 32 + kEpiThreads);
    }

    // ---------------------------------------------------- epilogue warps
    const int quad = warp & 3, group = (warp - 4) >> 2, row = quad * 32 + lane, et = tid - 128;
    const uint32_t trow = (uint32_t)(quad * 32) << 16;
    bool done = true, ok = true;
    float S_W = 0.f;
    const bool epi = warp >= 4 && warp < 12;
    // Row m0 + et's factor and span, from k_rows_prepare
    auto load_factors = [&](int buf) {
        const int parts = rows_parts(p.Ci);
        int span = 0;
        const float e = p.e[m0 + et];
        if (p.x_format != DQ_ROWS_E4M3)
            for (int i = 0; i < parts; i++) span += p.span[(m0 + et) * parts + i];
        bars.e[buf][et] = e;
        bars.span[buf][et] = span;
    };
    uint32_t used = 0;   // pieces so far
    // Rows that are not taken from their digits: their sums, ready before the accumulator is
    float4 wide[kPassRows / 8];
    bool any_wide = false;
    auto spans = [&](int b) { return *reinterpret_cast<const int4*>(&bars.span[used & 1][4 * b]); };
    auto form_wide = [&] {
        if (kFmt == DQ_ROWS_E4M3 || !ok) return;
        any_wide = false;
#pragma unroll 1
        for (int b = group; 4 * b < nm; b += 2) {
            const int4 s = spans(b);
            if (s.x > 0 || s.y > 0 || s.z > 0 || s.w > 0) {
                any_wide = true;
                wide[b >> 1] = (own ? wide_rows_call : wide_rows)(p.packed_w + p.off_codes, p.packed_w + p.off_scales, p.x, p.x_stride, p.x_scales, p.Ci,
                                         o0 + quad * 32, m0 + 4 * b, nm - 4 * b, a0 * 4, (a0 + nA) * 4, &bars.e[used & 1][4 * b]);
            }
        }
    };
    float bv = 0.f;
    if (own && warp < 4) cluster_wait();
    if (own && warp >= 12) lowrank_term<kFmt>(p, bars, up, su, slow, o0, crank, csize, split, splits);
    if (epi) {
        Raw8<kFmt> raw[kOwnTurns];
        if (own) load_own_rows<kFmt>(p, a0 * 256, nA * 256, raw);
        if (own) bar_arrive(3, 32 + 512);   // the weight may follow
        if (!pairs && warp < 8) {
            ones(t_one + trow);
            tc_fence_before();
            __syncwarp();
            bar_arrive(2, 32 + 128);
        }
        if (own) {
            write_own_digits<kFmt>(p, bars, digits, nA * 256, raw);
            cluster_wait();
        } else {
            griddep_wait();   // the rows' factors come from k_rows_prepare
            if (!pairs && et < nm) load_factors(0);
        }
        bar_sync(6, 32 + kEpiThreads);
        ok = bars.fits;
        S_W = bars.S_W;
        bv = bars.bias[row];
        if (!pairs) {
            bar_sync(1, kEpiThreads);
            form_wide();
            if (own) bar_sync(5, 512);   // the low-rank term
            if (lane == 0) done = mbar_wait(&bars.accf, 0, abort_flag, p.status, p.budget_ns);
            done = __shfl_sync(0xffffffffu, done && !*abort_flag, 0);   // (also where the low-rank term's wait ran out)
            tc_fence_after();
        }
    }
    // This CTA's part of the rows 4 b to 4 b + 3 for the thread's output channel: the digits' columns with
    // weights 8^-p, times S_W and the row's factor, and U L2 where this CTA has it
    auto parts_of = [&](int b, float (&v)[4]) {
        uint32_t acc[32], low[4];
        if (!own && split == 0) tmem_ld_x4(t_low + trow + (uint32_t)(4 * b), low);
#pragma unroll
        for (int c = 0; c < 32; c += 16) tmem_ld_x16(tmem + trow + (uint32_t)(32 * b + c), *reinterpret_cast<uint32_t(*)[16]>(&acc[c]));
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[i] = __uint_as_float(acc[kDigits * i + kDigits - 1]);
#pragma unroll
            for (int q = kDigits - 2; q >= 0; q--) v[i] = fmaf(v[i], 0.125f, __uint_as_float(acc[kDigits * i + q]));
        }
        if (kFmt != DQ_ROWS_E4M3 && (own || any_wide)) {
            const int4 s = spans(b);
            if (s.x > 0) v[0] = wide[b >> 1].x;
            if (s.y > 0) v[1] = wide[b >> 1].y;
            if (s.z > 0) v[2] = wide[b >> 1].z;
            if (s.w > 0) v[3] = wide[b >> 1].w;
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[i] = fmaf(v[i] * S_W, bars.e[used & 1][imin(4 * b + i, nm - 1)], !own && split == 0 ? __uint_as_float(low[i]) : 0.f);
    };
    // Y of the thread's output channel for the i-th of the rows split, split + splits, ... that this CTA finishes, and
    // for the next where there is one
    int mine = split < nm ? (nm - split + splits - 1) / splits : 0;
    auto finish = [&](int i, float y0, float y1) {
        const int m = split + i * splits;
        const bool two = i + 1 < mine;
        y0 += bv, y1 += bv;
        if (own) y0 += slow[i * 128 + row], y1 += two ? slow[(i + 1) * 128 + row] : 0.f;
        if (p.gelu) f2_unpack(gelu_erf2(f2_pack(y0, y1)), y0, y1);
        uint16_t* dst = p.y + (long long)(m0 + m) * p.y_stride + o0 + row;
        dst[0] = f32_to_bf16_rn(y0);
        if (two) dst[(long long)splits * p.y_stride] = f32_to_bf16_rn(y1);
    };
    if (pairs) {
        for (int item = item0; item < items && epi; item += step, used++) {
            o0 = tile_of(item), m0 = rows_of(item), mine = nm = imin(p.n_rows, p.rows - m0);
            if (used && ok && (bars.flags & kPackedHasBias)) bv = *(const float*)(p.packed_w + p.off_bias + 4ll * (o0 + row));
            if (et < nm) load_factors(used & 1);
            bar_sync(1, kEpiThreads);
            form_wide();
            // (a warp whose wait has run out goes on without writing, as the others still meet it at the barrier)
            bool full = true;
            if (lane == 0) full = mbar_wait(&bars.accf, used & 1, abort_flag, p.status, p.budget_ns);
            done = __shfl_sync(0xffffffffu, full && !*abort_flag, 0) && done;
            tc_fence_after();
            float v[kPassRows / 8][4];
#pragma unroll
            for (int k = 0; k < kPassRows / 8; k++)
                if (4 * (group + 2 * k) < nm) parts_of(group + 2 * k, v[k]);
            // the accumulator is free for the next piece
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&bars.acce), 0));
#pragma unroll
            for (int k = 0; k < kPassRows / 8; k++) {
                const int b = group + 2 * k;
                if (4 * b < nm && done && ok) {
                    finish(4 * b, v[k][0], v[k][1]);
                    if (4 * b + 2 < nm) finish(4 * b + 2, v[k][2], v[k][3]);
                }
            }
        }
    } else if (splits == 1) {
        if (epi && done && ok) {
            for (int b = group; 4 * b < nm; b += 2) {
                float v[4];
                parts_of(b, v);
                finish(4 * b, v[0], v[1]);
                if (4 * b + 2 < nm) finish(4 * b + 2, v[2], v[3]);
            }
        }
        __syncwarp();
        if (own) cluster_sync();   // no CTA leaves while another still reads its part of U
    } else {
        // The parts of a tile: the CTA of part r sums, in the order of the parts, the rows m with m % splits = r.
        // The buffer takes the operand ring's place, so every CTA of the cluster is past its MMAs first.
        __syncwarp();
        cluster_sync();
        float* red = (float*)sm;   // [part][row / splits][128 output channels]
        const int per = (nm + splits - 1) / splits, tile0 = crank - split;
        if (epi && done) {
            for (int b = group; 4 * b < nm; b += 2) {
                float v[4];
                parts_of(b, v);
                int dst = (4 * b) % splits, at = (4 * b) / splits;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (4 * b + i < nm)
                        st_dsmem_f32(mapa_shared(smem_u32(&red[(split * per + at) * 128 + row]), (uint32_t)(tile0 + dst)), v[i]);
                    if (++dst == splits) dst = 0, at++;
                }
            }
        }
        // without this CTA's part no CTA of the tile writes its rows
        if (epi && !done && lane < splits) st_dsmem_f32(mapa_shared(smem_u32(&bars.abort_flag), (uint32_t)(tile0 + lane)), 1.f);
        __syncwarp();
        cluster_sync();
        if (epi && done && ok && !*abort_flag) {
            for (int n = 2 * group; n < mine; n += 4) {
                float v0 = 0.f, v1 = 0.f;
                for (int q = 0; q < splits; q++) {
                    v0 += red[(q * per + n) * 128 + row];
                    if (n + 1 < mine) v1 += red[(q * per + n + 1) * 128 + row];
                }
                finish(n, v0, v1);
            }
        }
    }
    tc_fence_before();
    __syncwarp();
    if (pairs)
        cluster_sync();   // neither CTA leaves while the other may still touch its shared memory or barriers
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if (pairs)
            tmem_dealloc_pair(tmem, kTmemCols);
        else
            tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ host

// Runs `set` (a kernel's attributes) on the first call for that kernel on the current device.  Concurrent
// first calls may both run it; they set the same values.
template <typename Set>
cudaError_t once_per_device(const void* kernel, Set set) {
    constexpr int kKernels = 8, kDevices = 64;
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

// A call's two kernels; the product reads rows itself only when it writes their digits.
template <int kFmt, typename F>
auto by_form(const RowsParams& p, F f) {
    return p.own_digits ? f(k_rows_prepare<kFmt>, k_rows_product<kFmt, kOwnDigits>)
           : p.pairs    ? f(k_rows_prepare<kFmt>, k_rows_product<0, kPairs>)
                        : f(k_rows_prepare<kFmt>, k_rows_product<0, kPrepared>);
}

template <typename F>
auto by_format(const RowsParams& p, F f) {
    return p.x_format == DQ_ROWS_BF16   ? by_form<DQ_ROWS_BF16>(p, f)
           : p.x_format == DQ_ROWS_E4M3 ? by_form<DQ_ROWS_E4M3>(p, f)
                                        : by_form<DQ_ROWS_E4M3_GROUP64>(p, f);
}

template <typename K>
cudaError_t allow_smem(K kernel) {
    return once_per_device((const void*)kernel, [=] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    });
}

// Clusters of `size` CTAs of the product (one CTA per SM) that fit on the current device at once, the same for all
// forms; asked once per device and size.
cudaError_t resident_clusters(int size, int* clusters) {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][9];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    std::atomic<int>& k = known[dev][size];
    if ((*clusters = k.load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    auto kernel = k_rows_product<0, kPrepared>;
    if ((e = allow_smem(kernel)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)size, 1024);
    cfg.blockDim = dim3(product_threads(false));
    cfg.dynamicSmemBytes = kSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaOccupancyMaxActiveClusters(clusters, kernel, &cfg)) != cudaSuccess) return e;
    k.store(*clusters, std::memory_order_relaxed);
    return cudaSuccess;
}

// k_rows_prepare's clusters and CTAs (RowsParams' fields prep_*)
cudaError_t prepare_plan(RowsParams& p) {
    int sms = 0;
    cudaError_t e = resident_clusters(1, &sms);
    if (e != cudaSuccess) return e;
    // A CTA per row's piece and clusters of eight, while they are no more than four times what fits at once (64
    // registers a thread); else as many CTAs as fit, half of them low-rank ones at most, in smaller clusters, and
    // the others take piece after piece.  One CTA a piece against this: 5120 -> 5120 256 rows 39.8 us either way, 512 rows
    // 67 us against 58.5, 1024 rows 121 against 102; 256 rows 13824 -> 5120 85 us against 88, 512 rows 146 against 132;
    // 1024 rows 2048 -> 5120 59 us either way.  384 rows 5120 -> 5120, just below the bound, would take 46 us for 53.
    const long long fit = (long long)sms * (1024 / prep_threads(p.Ci)), groups = cdiv(p.rows, 16) * cdiv(p.rank, 32);
    long long pieces = (long long)p.rows * rows_parts(p.Ci);
    p.prep_cluster = kPrepCluster;
    if (groups * kPrepCluster + pieces > 4 * fit) {
        while (p.prep_cluster > 1 && groups * p.prep_cluster > fit / 2) p.prep_cluster /= 2;
        const long long rest = fit - groups * p.prep_cluster, most = rest >= fit / 4 ? rest : fit;
        if (pieces > most) pieces = most;
    }
    p.prep_ctas = (groups + cdiv(pieces, p.prep_cluster)) * p.prep_cluster;
    return cudaSuccess;
}

}  // namespace

// How the product of `rows` rows is cut (RowsParams' fields from n_rows on).
cudaError_t rows_plan(RowsParams& p) {
    p.passes = (int)cdiv(p.rows, kPassRows);
    p.n_rows = (int)cdiv(p.rows, p.passes);
    p.passes = (int)cdiv(p.rows, p.n_rows);
    p.n_pad = p.n_rows * kDigits;
    p.d_cols = (int)cdiv(p.n_pad, 32) * 32;
    const int tiles = p.Co / 128, k256 = p.Ci / 256;
    p.pairs = 0;
    for (int attempt = p.rows <= kOwnRows ? 0 : 1; attempt < 2; attempt++) {
        // up to kOwnRows rows the product does everything, if the digits and a ring of enough stages fit
        const bool own = attempt == 0;
        // a cluster splits the channels as far as every CTA is still resident at once; with the low-rank term
        // formed in it, it also takes as many tiles as fit, which then share the reading of L1
        p.splits = 1, p.group = 0;
        const int tries[] = {8, 6, 4, 3, 2, 1};
        for (int s : tries) {
            if (s > k256) continue;
            for (int g = own ? 8 / s : 1; g > 0 && !p.group; g--) {
                int clusters = 0;
                if (tiles % g) continue;
                cudaError_t e = resident_clusters(s * g, &clusters);
                if (e != cudaSuccess) return e;
                if (tiles / g * p.passes <= clusters) p.splits = s, p.group = g;
            }
            if (p.group) break;
        }
        if (!own && !p.group && p.passes > 2) {
            // more work than CTAs fit at once: CTA pairs that take piece after piece, the next one's operands under way
            // beside this one's output.  The passes (an even number of rows each: every CTA has half of the columns,
            // 64 of them to a kilobyte-aligned place) are cut so that the longest pair's rows are fewest.  With one or
            // two passes the weight's stream is the bound, which single CTAs keep up better: 5120 -> 13824, 48 rows
            // 30 us by pairs, 25 us by single CTAs; 96 rows (three passes) 31 us against 36 us; 5120 -> 5120, 512 rows
            // 57 us against 61 us (single CTAs, or pairs with one piece each: 63 us), 4096 rows 385 us against 440 us.
            p.pairs = 1, p.group = 2;
            int fit = 0;
            cudaError_t e = resident_clusters(2, &fit);
            if (e != cudaSuccess) return e;
            long long best = 0;
            for (int more = 0, least = p.passes; more < 4; more++) {
                const int n = ((int)cdiv(p.rows, least + more) + 1) & ~1, passes = (int)cdiv(p.rows, n);
                const long long longest = cdiv((long long)tiles / 2 * passes, fit) * n;
                if (more == 0 || longest < best) best = longest, p.n_rows = n, p.passes = passes;
            }
            p.pair_ctas = imin(fit, tiles / 2 * p.passes);
            p.n_pad = p.n_rows * kDigits;
            p.d_cols = (int)cdiv(p.n_pad, 32) * 32;
        }
        if (!p.group)   // more tiles than that: clusters of up to four of them for L1's sake
            for (p.group = own ? 4 : 1; tiles % p.group; p.group--) {
            }
        const int items = p.rank / 16, digits = p.n_pad * (p.pairs ? 64 : 128);
        p.u_parts = items < 8 ? 8 / items : 1;
        p.own_digits = own;
        p.own_stages = (int)cdiv(k256, p.splits);
        const int room = kSmem - 1024 - (own ? p.own_stages * digits + ((p.u_parts + 1) * 8 * p.rank + kOwnRows * 128) * 4 : 0);
        const int stage = (int)(kCodeBytes + kScaleBytes) + (own ? 0 : digits);
        p.stages = room < 0 ? 0 : imin(imin(kStages, room / stage), ((int)kTmemCols - p.d_cols - (int)cdiv(p.n_rows, 16) * 16 - 8) / 16);
        if (own && (p.stages < imin(6, p.own_stages) || p.own_stages > own_turns(p.rows) * own_warps(p.rows))) continue;
        break;
    }
    return p.own_digits ? cudaSuccess : prepare_plan(p);
}

cudaError_t launch_rows(const CUtensorMap& tm_w, const CUtensorMap& tm_s, const CUtensorMap& tm_x, const CUtensorMap& tm_l2,
                        const CUtensorMap& tm_u, const RowsParams& p, cudaStream_t st) {
    return by_format(p, [&](auto prepare, auto product) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.z = 1;
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        cudaError_t e;
        if (!p.own_digits) {
            // the product's split of the SM between L1 and shared memory: a different one would keep its CTAs off
            // an SM until this kernel's have left
            e = once_per_device((const void*)prepare, [&] {
                return cudaFuncSetAttribute(prepare, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
            });
            if (e != cudaSuccess) return e;
            attr[1].val.clusterDim.x = (unsigned)p.prep_cluster;
            attr[1].val.clusterDim.y = 1;
            cfg.gridDim = dim3((unsigned)p.prep_ctas);
            cfg.blockDim = dim3((unsigned)prep_threads(p.Ci));
            if ((e = cudaLaunchKernelEx(&cfg, prepare, p)) != cudaSuccess) return e;
        }
        if ((e = allow_smem(product)) != cudaSuccess) return e;
        if (p.pairs) {   // along x
            attr[1].val.clusterDim.x = 2;
            attr[1].val.clusterDim.y = 1;
            cfg.gridDim = dim3(2, (unsigned)p.pair_ctas);
        } else {
            attr[1].val.clusterDim.x = (unsigned)p.splits;
            attr[1].val.clusterDim.y = (unsigned)p.group;
            cfg.gridDim = dim3((unsigned)p.splits, (unsigned)(p.Co / 128), (unsigned)p.passes);
        }
        cfg.blockDim = dim3((unsigned)product_threads(p.own_digits != 0));
        cfg.dynamicSmemBytes = kSmem;
        return cudaLaunchKernelEx(&cfg, product, tm_w, tm_s, tm_x, tm_l2, tm_u, p);
    });
}

}  // namespace dq
