// fp8bq_fp4_quant.cu -- quantisation to microscaled 4-bit floating point
// (e2m1 codes with one scale for each run of values along a row) and back.
//
// MXFP4, 32 values a block: with a = max|x| of the block,
//     S = clamp(floor(log2 a) - 2, -127, 127)   (-127 for a = 0)
//     code = e2m1(x * 2^-S)                     to nearest even, beyond 6 to 6
// and the scale byte is S + 127 (e8m0).  The multiplication is exact, so the
// result is unique bit for bit (where it underflows, the code is 0 anyway).
//
// NVFP4, 16 values a block, t a positive fp32 scale of the whole tensor:
//     s = e4m3(min((a / 6) / t, 448))           IEEE fp32 divisions
//     d = s * t,  r = 1 / d (0 if d = 0)        each rounded to fp32, r finite
//     code = e2m1(x * r)                        the product rounded to fp32
//
// A block that holds an infinity or a NaN gets the NaN scale and zero codes.
// Values: code * scale (* t), one rounding at most before the output's own.
//
// Both passes are HBM-bound: 2 (4) bytes read and 0.53 (0.56) written an
// element one way, the reverse the other.
#include "fp8bq_device.cuh"
#include "fp8bq_fp4.h"

namespace fp8bq {
namespace {

#define FP4_SPAN_X(a) (dev::Span{(uint64_t)(a).x, (uint64_t)(a).x + (a).x_bytes})
#define FP4_SPAN_C(a) (dev::Span{(uint64_t)(a).codes, (uint64_t)(a).codes + (a).codes_bytes})
#define FP4_SPAN_S(a) (dev::Span{(uint64_t)(a).scales, (uint64_t)(a).scales + (a).scales_bytes})
#define FP4_SPAN_T(a) (dev::Span{(uint64_t)(a).tscale, (uint64_t)(a).tscale + (a).tscale_bytes})

template <int MAXD>
__device__ __forceinline__ int first_desc(const Fp4Pack<MAXD> &p, uint64_t k) {
    int lo = 0, hi = p.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.d[mid].begin <= k) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// A warp's work item: tile row (of the whole stack), row in it, run of COLS
// columns.
struct Item {
    int64_t b;          // matrix of the stack
    int64_t tile_row;   // over the stack
    int32_t row0;       // first of its four rows (32 apart), within the matrix
    int32_t r;          // row0 % 32
    int32_t seg;        // column run
};
template <int COLS>
__device__ __forceinline__ Item item_of(const Fp4Desc &a, uint64_t k) {
    const uint32_t segs = ((uint32_t)a.K + COLS - 1) / COLS;
    const uint64_t local = k - a.begin;
    Item it;
    uint64_t lr;
    if (a.items >> 32 == 0) {  // 32-bit divisions: a fifth of the 64-bit ones' instructions
        lr = (uint32_t)local / segs;
        it.b = (uint32_t)(lr >> 5) / (uint32_t)a.tiles_m;
    } else {
        lr = local / segs;
        it.b = (int64_t)((lr >> 5) / (uint32_t)a.tiles_m);
    }
    it.seg = (int32_t)(local - lr * segs);
    it.r = (int32_t)(lr & 31);
    it.tile_row = (int64_t)(lr >> 5);
    it.row0 = (int32_t)(it.tile_row - it.b * a.tiles_m) * kFp4TileRows + it.r;
    return it;
}

// ------------------------------------------------------------------ quantise

// A lane's N consecutive elements of a row (N * ES = 32 bytes), zero beyond
// `n`, bf16 two a word.  ALIGN: 32, 16 or 8, which every row is aligned to.
// With less than 32 the lane's accesses share sectors, which L1 then keeps.
template <int ES, int ALIGN>
__device__ __forceinline__ void load32(const char *p, int n, uint32_t (&v)[8],
                                       [[maybe_unused]] const dev::Span &xs) {
    constexpr int N = 32 / ES;
    if (n >= N) {
        if (!FP8BQ_IN(xs, p, 32)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0;
        } else if constexpr (ALIGN == 32) {
            asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v8.b32 "
                         "{%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                           "=r"(v[6]), "=r"(v[7])
                         : "l"(p));
        } else if constexpr (ALIGN == 16) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 q = __ldg((const uint4 *)(p + 16 * i));
                v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint2 q = dev::ldg_v2(p + 8 * i);
                v[2 * i] = q.x, v[2 * i + 1] = q.y;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n && FP8BQ_IN(xs, p + i * ES, ES)) {
                if constexpr (ES == 2)
                    v[i / 2] |= (uint32_t)__ldg((const unsigned short *)p + i) << (16 * (i & 1));
                else
                    v[i] = __float_as_uint(__ldg((const float *)p + i));
            }
    }
}

// The same for rows of any alignment: the warp's 1024 bytes by element, so
// that a load instruction covers consecutive addresses, through shared memory.
template <int ES>
__device__ __forceinline__ void load_by_element(const char *row, int lane, int n, char *buf,
                                                [[maybe_unused]] const dev::Span &xs) {
#pragma unroll
    for (int j = 0; j < 32 / ES; ++j) {
        const int c = 32 * j + lane;
        const bool in = c < n && FP8BQ_IN(xs, row + c * ES, ES);
        if constexpr (ES == 2)
            *(unsigned short *)(buf + 2 * c) = in ? __ldg((const unsigned short *)row + c) : 0;
        else
            *(float *)(buf + 4 * c) = in ? __ldg((const float *)row + c) : 0.0f;
    }
}

// Running maxima of magnitudes that keep a NaN (the sign bit means nothing).
__device__ __forceinline__ uint32_t amax_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t amax_f32(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Eight codes of x * r, element 0 in the low four bits.
__device__ __forceinline__ uint32_t codes8(uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3,
                                           uint32_t v4, uint32_t v5, uint32_t v6, uint32_t v7,
                                           float r) {
    uint32_t o;
    asm("{\n\t.reg .b64 rr, a, b, c, d;\n\t.reg .f32 l, h;\n\t.reg .b8 p, q, s, t;\n\t"
        "mov.b64 rr, {%9, %9};\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "mov.b64 c, {%5, %6};\n\tmov.b64 d, {%7, %8};\n\t"
        "mul.rn.f32x2 a, a, rr;\n\tmul.rn.f32x2 b, b, rr;\n\t"
        "mul.rn.f32x2 c, c, rr;\n\tmul.rn.f32x2 d, d, rr;\n\t"
        "mov.b64 {l, h}, a;\n\tcvt.rn.satfinite.e2m1x2.f32 p, h, l;\n\t"
        "mov.b64 {l, h}, b;\n\tcvt.rn.satfinite.e2m1x2.f32 q, h, l;\n\t"
        "mov.b64 {l, h}, c;\n\tcvt.rn.satfinite.e2m1x2.f32 s, h, l;\n\t"
        "mov.b64 {l, h}, d;\n\tcvt.rn.satfinite.e2m1x2.f32 t, h, l;\n\t"
        "mov.b32 %0, {p, q, s, t};\n\t}"
        : "=r"(o)
        : "r"(v0), "r"(v1), "r"(v2), "r"(v3), "r"(v4), "r"(v5), "r"(v6), "r"(v7), "f"(r));
    return o;
}
// The codes of a lane's 32 bytes: 16 bf16 (two words of codes) or 8 fp32 (one).
__device__ __forceinline__ uint32_t codes_bf16(const uint32_t *w, float r) {
    return codes8(w[0] << 16, w[0] & 0xffff0000u, w[1] << 16, w[1] & 0xffff0000u, w[2] << 16,
                  w[2] & 0xffff0000u, w[3] << 16, w[3] & 0xffff0000u, r);
}

// Scale byte and multiplier of a block from the bits of its absmax; -0 as the
// multiplier of a block that is not finite.
template <int FMT>
__device__ __forceinline__ uint32_t block_scale4(uint32_t amax, float t, float &r) {
    const bool bad = amax >= 0x7f800000u;
    uint32_t s;
    if constexpr (FMT == FP8BQ_MXFP4) {
        const uint32_t e = amax >> 23;              // 0 for zero and subnormals
        s = e > 2 ? e - 2 : 0;                      // S + 127
        r = __uint_as_float((254u - s) << 23);      // 2^(127 - s), 2^-125 at least
    } else {
        const float want = fminf(__fdiv_rn(__fdiv_rn(__uint_as_float(amax), 6.0f), t), 448.0f);
        s = dev::cvt_e4m3x2(want, 0.0f) & 0xffu;
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)s));
        float f;
        asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}"
            : "=f"(f) : "r"(h2));
        const float d = __fmul_rn(f, t);
        r = d > 0.0f ? fminf(__frcp_rn(d), 3.402823466e38f) : 0.0f;
    }
    if (bad) r = -0.0f;
    return bad ? (FMT == FP8BQ_MXFP4 ? 0xffu : 0x7fu) : s;
}

// A lane holds 32 bytes of each of its four rows, so a block is LPB = 1, 2 or
// 4 lanes of a row.  Where it is more than one, the rows' maxima are reduced
// and handed out at once: each lane of a block ends with the block's maximum
// in R = 4 / LPB of the rows (rows R (lane % LPB) and the next), finds those
// scales alone and passes the multipliers on.  The scale bytes of a tile's
// four blocks are then joined into the words of its rows in the tile's
// 16-byte run.
//
// Measured on B200, 12288 x 4096 bf16: mxfp4 20.5 us (6.2 TB/s), nvfp4 23.0
// (5.6; 25.3 with three CTAs an SM, 24.4 with five); 65536 x 4096 mxfp4 98.6
// (6.9 TB/s).  16 bytes a lane and row: 23.7, 30.3, 115.8; every lane reducing
// and scaling all four rows as well: 39.
template <int FMT, int ES, int ALIGN, int MAXD>
__global__ void __launch_bounds__(256, 4) k_fp4_quant(const __grid_constant__ Fp4Pack<MAXD> p) {
    dev::pdl_entry();
    constexpr int N = 32 / ES;                         // elements of a lane
    constexpr int LPB = fp4_block(FMT) / N;            // lanes a block
    constexpr int R = 4 / LPB;                         // rows whose scales a lane finds
    constexpr int TL = 4 * LPB;                        // lanes a tile
    constexpr bool kByElement = ALIGN < 8;
    __shared__ __align__(16) char stage[kByElement ? 8 : 1][4][kByElement ? 1024 : 16];
    const int lane = threadIdx.x & 31;
    const uint64_t warps = (uint64_t)gridDim.x * (blockDim.x >> 5);
    const uint64_t k0 = (uint64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    int d = k0 < p.total ? first_desc(p, k0) : 0;
    for (uint64_t k = k0; k < p.total; k += warps) {
        while (k >= p.d[d].begin + p.d[d].items) ++d;
        const Fp4Desc &a = p.d[d];
        const Item it = item_of<32 * N>(a, k);
        const int s0 = it.seg * 32 * N, c0 = s0 + lane * N;
        const int n = a.K - c0;                        // columns of this lane that exist
        const int64_t kb = (int64_t)((a.K + 31) >> 5) * 16;
#if FP8BQ_CHECKED
        const dev::Span xs = FP4_SPAN_X(a);
#else
        constexpr dev::Span xs{0, 0};
#endif
        uint32_t v[4][8];
        if constexpr (kByElement) {
            const char *x = (const char *)a.x + (it.b * a.xbs + it.row0 * a.ld + s0) * ES;
            char(*buf)[1024] = stage[threadIdx.x >> 5];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                load_by_element<ES>(x + (int64_t)(32 * i) * a.ld * ES, lane,
                                    it.row0 + 32 * i < a.M ? a.K - s0 : 0, buf[i], xs);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 q = *(const uint4 *)(buf[i] + lane * 32 + 16 * j);
                    v[i][4 * j] = q.x, v[i][4 * j + 1] = q.y;
                    v[i][4 * j + 2] = q.z, v[i][4 * j + 3] = q.w;
                }
            __syncwarp();
        } else {
            const char *x = (const char *)a.x + (it.b * a.xbs + it.row0 * a.ld + c0) * ES;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                load32<ES, ALIGN>(x + (int64_t)(32 * i) * a.ld * ES,
                                  it.row0 + 32 * i < a.M ? n : 0, v[i], xs);
        }
        float t = 1.0f;
        if (FMT == FP8BQ_NVFP4 && a.tscale != nullptr &&
            FP8BQ_IN(FP4_SPAN_T(a), a.tscale + it.b * a.tbs, 4))
            t = __ldg(a.tscale + it.b * a.tbs);

        // m[h], h < R: the block's maximum (fp32 bits) in row R (lane % LPB) + h
        uint32_t m[4];
        if constexpr (ES == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                m[i] = amax_bf16x2(amax_bf16x2(amax_bf16x2(v[i][0], v[i][1]),
                                               amax_bf16x2(v[i][2], v[i][3])),
                                   amax_bf16x2(amax_bf16x2(v[i][4], v[i][5]),
                                               amax_bf16x2(v[i][6], v[i][7])));
            uint32_t lo =
                amax_bf16x2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
            const uint32_t hi =
                amax_bf16x2(__byte_perm(m[2], m[3], 0x5410), __byte_perm(m[2], m[3], 0x7632));
            if constexpr (LPB == 2) {
                const bool up = lane & 1;              // keeps rows 2 and 3
                lo = amax_bf16x2(up ? hi : lo, __shfl_xor_sync(0xffffffffu, up ? lo : hi, 1));
            }
            m[0] = (lo << 16) & 0x7fffffffu;
            m[1] = lo & 0x7fff0000u;
            m[2] = (hi << 16) & 0x7fffffffu;
            m[3] = hi & 0x7fff0000u;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                m[i] = amax_f32(amax_f32(amax_f32(v[i][0], v[i][1]), amax_f32(v[i][2], v[i][3])),
                                amax_f32(amax_f32(v[i][4], v[i][5]), amax_f32(v[i][6], v[i][7])));
            const bool up = lane & (LPB / 2);
            const uint32_t g0 = __shfl_xor_sync(0xffffffffu, up ? m[0] : m[2], LPB / 2);
            const uint32_t g1 = __shfl_xor_sync(0xffffffffu, up ? m[1] : m[3], LPB / 2);
            m[0] = amax_f32(up ? m[2] : m[0], g0);
            m[1] = amax_f32(up ? m[3] : m[1], g1);
            if constexpr (LPB == 4) {
                const uint32_t g = __shfl_xor_sync(0xffffffffu, (lane & 1) ? m[0] : m[1], 1);
                m[0] = amax_f32((lane & 1) ? m[1] : m[0], g);
            }
            m[0] &= 0x7fffffffu;
            m[1] &= 0x7fffffffu;
        }
        uint32_t s[R];
        float mine[R], r[4];
#pragma unroll
        for (int h = 0; h < R; ++h) s[h] = block_scale4<FMT>(m[h], t, mine[h]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = LPB == 1 ? mine[i % R]
                            : __shfl_sync(0xffffffffu, mine[i % R], lane - lane % LPB + i / R);

        uint8_t *codes = a.codes + (it.b * a.M + it.row0) * kb + (c0 >> 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // a block that is not finite: inf * 0 would be NaN
            const uint32_t keep = __float_as_uint(r[i]) == 0x80000000u ? 0u : ~0u;
            uint8_t *dst = codes + (int64_t)(32 * i) * kb;
            const bool in = it.row0 + 32 * i < a.M && c0 < 2 * kb && FP8BQ_IN(FP4_SPAN_C(a), dst, N / 2);
            if constexpr (ES == 2) {
                const uint2 c = make_uint2(codes_bf16(v[i], r[i]) & keep,
                                           codes_bf16(v[i] + 4, r[i]) & keep);
                if (in) dev::stg_stream_v2(dst, c);
            } else {
                const uint32_t c = codes8(v[i][0], v[i][1], v[i][2], v[i][3], v[i][4], v[i][5],
                                          v[i][6], v[i][7], r[i]) & keep;
                if (in) dev::stg_stream_u32(dst, c);
            }
        }

        const int blk = (lane % TL) / LPB;
        const int tile = it.seg * (32 / TL) + lane / TL;
        const int i0 = lane % LPB * R;                 // this lane's first row
        uint8_t *run = a.scales + (it.tile_row * a.tiles_k + tile) * kFp4TileBytes + it.r * 16;
        const bool exists = (c0 & ~(N * LPB - 1)) < a.K;   // the block's first column does
#pragma unroll
        for (int h = 0; h < R; ++h)
            if (!exists || it.row0 + 32 * (i0 + h) >= a.M) s[h] = 0;
        if constexpr (LPB == 1) {  // a 4 x 4 transpose of bytes: lane `blk` gets row blk's word
            const uint32_t q = s[0] | s[1 % R] << 8 | s[2 % R] << 16 | s[3 % R] << 24;
            const uint32_t q2 = __shfl_xor_sync(0xffffffffu, q, 2);
            const uint32_t u = (lane & 2) ? __byte_perm(q2, q, 0x7632) : __byte_perm(q, q2, 0x5410);
            const uint32_t u2 = __shfl_xor_sync(0xffffffffu, u, 1);
            const uint32_t w = (lane & 1) ? __byte_perm(u2, u, 0x7351) : __byte_perm(u, u2, 0x6240);
            if (tile < a.tiles_k && FP8BQ_IN(FP4_SPAN_S(a), run + 4 * blk, 4))
                *(uint32_t *)(run + 4 * blk) = w;
        } else {
            uint32_t w[R];
#pragma unroll
            for (int h = 0; h < R; ++h) {
                w[h] = s[h] << (8 * blk);
#pragma unroll
                for (int o = LPB; o < TL; o *= 2) w[h] |= __shfl_xor_sync(0xffffffffu, w[h], o);
            }
            if (blk == 0 && tile < a.tiles_k && FP8BQ_IN(FP4_SPAN_S(a), run + 4 * i0, 4 * R)) {
                if constexpr (R == 1) *(uint32_t *)(run + 4 * i0) = w[0];
                else *(uint2 *)(run + 4 * i0) = make_uint2(w[0], w[1 % R]);
            }
        }
    }
}

// ------------------------------------------------------------------ dequantise

// Four values of two code bytes.
__device__ __forceinline__ void decode4(uint32_t c, float &v0, float &v1, float &v2, float &v3) {
    uint32_t h0, h1;
    asm("{\n\t.reg .b8 a, b, x, y;\n\t"
        "mov.b32 {a, b, x, y}, %2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t}"
        : "=r"(h0), "=r"(h1)
        : "r"(c));
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(v0), "=f"(v1) : "r"(h0));
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(v2), "=f"(v3) : "r"(h1));
}

template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t s) {
    if constexpr (FMT == FP8BQ_MXFP4) {
        return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7fffffffu : s << 23);
    } else {
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)s));
        float f;
        asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}"
            : "=f"(f) : "r"(h2));
        return f;
    }
}

// Rows that are not 32-byte aligned pass through shared memory: the warp's
// 1024 bytes go out in pieces of W bytes, piece j * 32 + lane by lane, so that
// a store instruction covers consecutive addresses and fills its sectors.
template <int W> struct Piece;
template <> struct Piece<16> { using T = uint4; };
template <> struct Piece<8> { using T = uint2; };
template <> struct Piece<4> { using T = uint32_t; };
template <> struct Piece<2> { using T = uint16_t; };

template <int OES, int W>
__device__ __forceinline__ void stage_to_row(const char *buf, int lane, int n, char *row,
                                             [[maybe_unused]] const dev::Span &xs) {
    using P = typename Piece<W>::T;
    constexpr int E = W / OES;
#pragma unroll
    for (int j = 0; j < 32 / W; ++j) {
        const int c = (32 * j + lane) * E;
        if (c + E <= n) {
            if (FP8BQ_IN(xs, row + c * OES, W)) *(P *)(row + c * OES) = *(const P *)(buf + c * OES);
        } else {
#pragma unroll
            for (int q = 0; q < E; ++q)
                if (c + q < n && FP8BQ_IN(xs, row + (c + q) * OES, OES)) {
                    if constexpr (OES == 2)
                        *(uint16_t *)(row + 2 * (c + q)) = *(const uint16_t *)(buf + 2 * (c + q));
                    else
                        *(uint32_t *)(row + 4 * (c + q)) = *(const uint32_t *)(buf + 4 * (c + q));
                }
        }
    }
}

// ALIGN: bytes (32, 16, 8, or the element's) that every output row is aligned
// to.
template <int FMT, int OES, int ALIGN, int MAXD>
__global__ void __launch_bounds__(256) k_fp4_dequant(const __grid_constant__ Fp4Pack<MAXD> p) {
    dev::pdl_entry();
    constexpr int N = 32 / OES;                        // outputs of a lane
    constexpr int LPB = fp4_block(FMT) / N;
    constexpr int TL = 4 * LPB;
    constexpr bool kStaged = ALIGN < 32;
    __shared__ __align__(16) char stage[kStaged ? 8 : 1][kStaged ? 1024 : 16];
    const int lane = threadIdx.x & 31;
    const uint64_t warps = (uint64_t)gridDim.x * (blockDim.x >> 5);
    const uint64_t k0 = (uint64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    int d = k0 < p.total ? first_desc(p, k0) : 0;
    for (uint64_t k = k0; k < p.total; k += warps) {
        while (k >= p.d[d].begin + p.d[d].items) ++d;
        const Fp4Desc &a = p.d[d];
        const Item it = item_of<32 * N>(a, k);
        const int c0 = it.seg * 32 * N + lane * N;
        const int n = a.K - c0;
        const int64_t kb = (int64_t)((a.K + 31) >> 5) * 16;
        const uint8_t *codes = a.codes + (it.b * a.M + it.row0) * kb + (c0 >> 1);
        uint32_t q[4][N / 8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t *src = codes + (int64_t)(32 * i) * kb;
#pragma unroll
            for (int j = 0; j < N / 8; ++j) q[i][j] = 0;
            if (n > 0 && it.row0 + 32 * i < a.M && FP8BQ_IN(FP4_SPAN_C(a), src, N / 2)) {
                if constexpr (N == 16)
                    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                                 : "=r"(q[i][0]), "=r"(q[i][1]) : "l"(src));
                else
                    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];"
                                 : "=r"(q[i][0]) : "l"(src));
            }
        }
        const int tile = it.seg * (32 / TL) + lane / TL, blk = (lane % TL) / LPB;
        const uint8_t *run =
            a.scales + (it.tile_row * a.tiles_k + tile) * kFp4TileBytes + it.r * 16;
        uint4 sw = make_uint4(0u, 0u, 0u, 0u);
        if (n > 0 && FP8BQ_IN(FP4_SPAN_S(a), run, 16)) sw = __ldg((const uint4 *)run);
        const uint32_t sv[4] = {sw.x, sw.y, sw.z, sw.w};
        float t = 1.0f;
        if (FMT == FP8BQ_NVFP4 && a.tscale != nullptr &&
            FP8BQ_IN(FP4_SPAN_T(a), a.tscale + it.b * a.tbs, 4))
            t = __ldg(a.tscale + it.b * a.tbs);
#if FP8BQ_CHECKED
        const dev::Span os = FP4_SPAN_X(a);
#else
        constexpr dev::Span os{0, 0};
#endif
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (it.row0 + 32 * i >= a.M) break;        // the same for the whole warp
            const float s = scale_value<FMT>((sv[i] >> (8 * blk)) & 0xffu);
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < N / 4; ++j) {
                float v[4];
                decode4(q[i][j / 2] >> (16 * (j & 1)), v[0], v[1], v[2], v[3]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = __fmul_rn(v[e], s);         // exact
                    if (FMT == FP8BQ_NVFP4) v[e] = __fmul_rn(v[e], t);
                    if (OES == 4) o[(4 * j + e) & 7] = __float_as_uint(v[e]);
                }
                if constexpr (OES == 2) {
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[2 * j]) : "f"(v[1]), "f"(v[0]));
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[2 * j + 1]) : "f"(v[3]), "f"(v[2]));
                }
            }
            char *dst = (char *)const_cast<void *>(a.x) +
                        (it.b * a.xbs + (int64_t)(it.row0 + 32 * i) * a.ld + c0) * OES;
            if constexpr (kStaged) {
                char *buf = stage[threadIdx.x >> 5];
                *(uint4 *)(buf + lane * 32) = make_uint4(o[0], o[1], o[2], o[3]);
                *(uint4 *)(buf + lane * 32 + 16) = make_uint4(o[4], o[5], o[6], o[7]);
                __syncwarp();
                stage_to_row<OES, ALIGN>(buf, lane, a.K - it.seg * 32 * N, dst - lane * 32, os);
                __syncwarp();
            } else if (n >= N) {
                if (FP8BQ_IN(os, dst, 32))
                    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst),
                                 "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]),
                                 "r"(o[6]), "r"(o[7])
                                 : "memory");
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (j < n && FP8BQ_IN(os, dst + j * OES, OES)) {
                        if constexpr (OES == 2)
                            *(uint16_t *)(dst + 2 * j) = (uint16_t)(o[j / 2] >> (16 * (j & 1)));
                        else
                            *(uint32_t *)(dst + 4 * j) = o[j];
                    }
            }
        }
    }
}

unsigned fp4_grid(uint64_t items, int per_sm) {  // a warp an item, 8 warps a CTA
    const uint64_t need = (items + 7) / 8;
    const uint64_t cap = (uint64_t)sm_count() * per_sm;
    return (unsigned)(need < 1 ? 1 : need < cap ? need : cap);
}

// Grid cap.  Measured on B200, 12288 x 4096 bf16 and 65536 x 4096: 16 a SM
// 2-4 % slower, 64 and more within 1 % either way.
constexpr int kFp4CtasPerSm = 32;

template <typename K, typename P>
cudaError_t launch_fp4(bool overlap, K kern, unsigned grid, cudaStream_t st, const P &p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = 256;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int FMT, int ES, int MAXD>
cudaError_t quant_align(const Fp4Pack<MAXD> &p, int align, bool overlap, cudaStream_t st) {
    const unsigned grid = fp4_grid(p.total, kFp4CtasPerSm);
    if (align >= 32) return launch_fp4(overlap, k_fp4_quant<FMT, ES, 32, MAXD>, grid, st, p);
    if (align >= 16) return launch_fp4(overlap, k_fp4_quant<FMT, ES, 16, MAXD>, grid, st, p);
    if (align >= 8) return launch_fp4(overlap, k_fp4_quant<FMT, ES, 8, MAXD>, grid, st, p);
    return launch_fp4(overlap, k_fp4_quant<FMT, ES, ES, MAXD>, grid, st, p);
}

template <int FMT, int OES, int MAXD>
cudaError_t dequant_align(const Fp4Pack<MAXD> &p, int align, bool overlap, cudaStream_t st) {
    const unsigned grid = fp4_grid(p.total, kFp4CtasPerSm);
    if (align >= 32) return launch_fp4(overlap, k_fp4_dequant<FMT, OES, 32, MAXD>, grid, st, p);
    if (align >= 16) return launch_fp4(overlap, k_fp4_dequant<FMT, OES, 16, MAXD>, grid, st, p);
    if (align >= 8) return launch_fp4(overlap, k_fp4_dequant<FMT, OES, 8, MAXD>, grid, st, p);
    return launch_fp4(overlap, k_fp4_dequant<FMT, OES, OES, MAXD>, grid, st, p);
}

}  // namespace

template <int MAXD>
cudaError_t launch_fp4_quantize(const Fp4Pack<MAXD> &p, int format, int esize, int align,
                                bool overlap, cudaStream_t st) {
    if (format == FP8BQ_MXFP4)
        return esize == 2 ? quant_align<FP8BQ_MXFP4, 2>(p, align, overlap, st)
                          : quant_align<FP8BQ_MXFP4, 4>(p, align, overlap, st);
    return esize == 2 ? quant_align<FP8BQ_NVFP4, 2>(p, align, overlap, st)
                      : quant_align<FP8BQ_NVFP4, 4>(p, align, overlap, st);
}

template <int MAXD>
cudaError_t launch_fp4_dequantize(const Fp4Pack<MAXD> &p, int format, int esize, int align,
                                  bool overlap, cudaStream_t st) {
    if (format == FP8BQ_MXFP4)
        return esize == 2 ? dequant_align<FP8BQ_MXFP4, 2>(p, align, overlap, st)
                          : dequant_align<FP8BQ_MXFP4, 4>(p, align, overlap, st);
    return esize == 2 ? dequant_align<FP8BQ_NVFP4, 2>(p, align, overlap, st)
                      : dequant_align<FP8BQ_NVFP4, 4>(p, align, overlap, st);
}

template cudaError_t launch_fp4_quantize<kMaxDescSmall>(const Fp4Pack<kMaxDescSmall> &, int, int,
                                                        int, bool, cudaStream_t);
template cudaError_t launch_fp4_quantize<kMaxFp4Large>(const Fp4Pack<kMaxFp4Large> &, int, int, int,
                                                       bool, cudaStream_t);
template cudaError_t launch_fp4_dequantize<kMaxDescSmall>(const Fp4Pack<kMaxDescSmall> &, int, int,
                                                          int, bool, cudaStream_t);

FP8BQ_DEFINE_BOUNDS_RECORD(bounds_record_fp4_quant)

}  // namespace fp8bq
