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
//     d = s * t,  r = 1 / d (0 if d = 0)        each rounded to fp32
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

// A warp's work item: tile row (of the whole stack), row in it, column run.
struct Item {
    int64_t b;          // matrix of the stack
    int64_t tile_row;   // over the stack
    int32_t row0;       // first of its four rows (32 apart), within the matrix
    int32_t r;          // row0 % 32
    int32_t seg;        // 256-column run
};
__device__ __forceinline__ Item item_of(const Fp4Desc &a, uint64_t k) {
    const uint32_t segs = (uint32_t)((a.K + kFp4ItemCols - 1) / kFp4ItemCols);
    const uint64_t local = k - a.begin;
    const uint64_t lr = local / segs;
    Item it;
    it.seg = (int32_t)(local - lr * segs);
    it.r = (int32_t)(lr & 31);
    it.tile_row = (int64_t)(lr >> 5);
    it.b = it.tile_row / a.tiles_m;
    it.row0 = (int32_t)((it.tile_row - it.b * a.tiles_m) * kFp4TileRows) + it.r;
    return it;
}

// ------------------------------------------------------------------ quantise

// Eight consecutive elements of a row as fp32 bit patterns, zero beyond `n`.
// ALIGN: bytes of the widest load its address allows.
template <int ES, int ALIGN>
__device__ __forceinline__ void load8(const char *p, int n, uint32_t (&v)[8],
                                      [[maybe_unused]] const dev::Span &xs) {
    if (n >= 8 && ALIGN >= 8) {
        uint32_t w[2 * ES];
        if constexpr (ALIGN == 16) {
#pragma unroll
            for (int i = 0; i < ES / 2; ++i) {
                const uint4 q = FP8BQ_IN(xs, p + 16 * i, 16) ? dev::ldg_stream_v4(p + 16 * i)
                                                             : make_uint4(0u, 0u, 0u, 0u);
                w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < ES; ++i) {
                const uint2 q = FP8BQ_IN(xs, p + 8 * i, 8) ? dev::ldg_v2(p + 8 * i)
                                                           : make_uint2(0u, 0u);
                w[2 * i] = q.x, w[2 * i + 1] = q.y;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (ES == 2) v[i] = (i & 1) ? w[i / 2] & 0xffff0000u : w[i / 2] << 16;
            else v[i] = w[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = 0;
            if (i < n && FP8BQ_IN(xs, p + i * ES, ES)) {
                if constexpr (ES == 2) v[i] = (uint32_t)__ldg((const unsigned short *)p + i) << 16;
                else v[i] = __float_as_uint(__ldg((const float *)p + i));
            }
        }
    }
}

// Eight codes of x * r, element 0 in the low four bits.
__device__ __forceinline__ uint32_t codes8(const uint32_t (&v)[8], float r) {
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
        : "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
          "f"(r));
    return o;
}

// Scale byte and multiplier of a block from the bits of its absmax.
template <int FMT>
__device__ __forceinline__ uint32_t block_scale4(uint32_t amax, float t, float &r) {
    const bool bad = amax >= 0x7f800000u;
    if constexpr (FMT == FP8BQ_MXFP4) {
        const uint32_t e = amax >> 23;              // 0 for zero and subnormals
        const uint32_t s = e > 2 ? e - 2 : 0;       // S + 127
        r = __uint_as_float((254u - s) << 23);      // 2^(127 - s), 2^2 at least
        if (bad) r = 0.0f;
        return bad ? 0xffu : s;
    } else {
        const float want = fminf(__fdiv_rn(__fdiv_rn(__uint_as_float(amax), 6.0f), t), 448.0f);
        const uint32_t s = dev::cvt_e4m3x2(want, 0.0f) & 0xffu;
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)s));
        float f;
        asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}"
            : "=f"(f) : "r"(h2));
        const float d = __fmul_rn(f, t);
        r = d > 0.0f && !bad ? fminf(__frcp_rn(d), 3.402823466e38f) : 0.0f;
        return bad ? 0x7fu : s;
    }
}

template <int FMT, int ES, int ALIGN, int MAXD>
__global__ void __launch_bounds__(256) k_fp4_quant(const __grid_constant__ Fp4Pack<MAXD> p) {
    dev::pdl_entry();
    constexpr int LPB = FMT == FP8BQ_MXFP4 ? 4 : 2;    // lanes a block
    const int lane = threadIdx.x & 31;
    const uint64_t warps = (uint64_t)gridDim.x * (blockDim.x >> 5);
    const uint64_t k0 = (uint64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    int d = k0 < p.total ? first_desc(p, k0) : 0;
    for (uint64_t k = k0; k < p.total; k += warps) {
        while (k >= p.d[d].begin + p.d[d].items) ++d;
        const Fp4Desc &a = p.d[d];
        const Item it = item_of(a, k);
        const int c0 = it.seg * kFp4ItemCols + lane * 8;
        const int n = a.K - c0;                        // columns of this lane that exist
        const int64_t kb = (int64_t)((a.K + 31) >> 5) * 16;
#if FP8BQ_CHECKED
        const dev::Span xs = FP4_SPAN_X(a);
#else
        constexpr dev::Span xs{0, 0};
#endif
        const char *x = (const char *)a.x + (it.b * a.xbs + it.row0 * a.ld + c0) * ES;
        uint32_t v[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = it.row0 + 32 * i < a.M;
            load8<ES, ALIGN>(x + (int64_t)(32 * i) * a.ld * ES, in ? n : 0, v[i], xs);
        }
        float t = 1.0f;
        if (FMT == FP8BQ_NVFP4 && a.tscale != nullptr &&
            FP8BQ_IN(FP4_SPAN_T(a), a.tscale + it.b * a.tbs, 4))
            t = __ldg(a.tscale + it.b * a.tbs);
        uint8_t *codes = a.codes + (it.b * a.M + it.row0) * kb + (c0 >> 1);
        uint32_t s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, v[i][j] & 0x7fffffffu);
#pragma unroll
            for (int o = 1; o < LPB; o *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            float r;
            s[i] = block_scale4<FMT>(m, t, r);
            const bool in = it.row0 + 32 * i < a.M;
            if (!in) s[i] = 0;
            const bool bad = m >= 0x7f800000u;         // inf * 0 would be NaN
            const uint32_t c = bad ? 0u : codes8(v[i], r);
            uint8_t *dst = codes + (int64_t)(32 * i) * kb;
            if (in && c0 < 2 * kb && FP8BQ_IN(FP4_SPAN_C(a), dst, 4)) dev::stg_stream_u32(dst, c);
        }
        // Word i of a tile's 16-byte run holds the four blocks of row i: a
        // lane takes row(s) by its place in the block and the words are
        // joined over the blocks.
        constexpr int TL = 4 * LPB;                    // lanes a tile
        const int blk = (lane % TL) / LPB;
        const int tile = it.seg * (32 / TL) + lane / TL;
        uint8_t *run = a.scales + (it.tile_row * a.tiles_k + tile) * kFp4TileBytes + it.r * 16;
#pragma unroll
        for (int h = 0; h < 4 / LPB; ++h) {
            const int i = lane % LPB + LPB * h;
            uint32_t w = s[0];
#pragma unroll
            for (int q = 1; q < 4; ++q) w = i == q ? s[q] : w;
            // columns beyond K: the lane of the block's first column decides
            w = __shfl_sync(0xffffffffu, n > 0, lane - lane % LPB) ? w : 0u;
            w <<= 8 * blk;
#pragma unroll
            for (int o = LPB; o < TL; o *= 2) w |= __shfl_xor_sync(0xffffffffu, w, o);
            if (blk == 0 && tile < a.tiles_k && FP8BQ_IN(FP4_SPAN_S(a), run + 4 * i, 4))
                *(uint32_t *)(run + 4 * i) = w;
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

template <int FMT, int OES, bool VEC, int MAXD>
__global__ void __launch_bounds__(256) k_fp4_dequant(const __grid_constant__ Fp4Pack<MAXD> p) {
    dev::pdl_entry();
    constexpr int LPB = FMT == FP8BQ_MXFP4 ? 4 : 2;
    constexpr int TL = 4 * LPB;
    const int lane = threadIdx.x & 31;
    const uint64_t warps = (uint64_t)gridDim.x * (blockDim.x >> 5);
    const uint64_t k0 = (uint64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    int d = k0 < p.total ? first_desc(p, k0) : 0;
    for (uint64_t k = k0; k < p.total; k += warps) {
        while (k >= p.d[d].begin + p.d[d].items) ++d;
        const Fp4Desc &a = p.d[d];
        const Item it = item_of(a, k);
        const int c0 = it.seg * kFp4ItemCols + lane * 8;
        const int n = a.K - c0;
        if (n <= 0) continue;
        const int64_t kb = (int64_t)((a.K + 31) >> 5) * 16;
        const uint8_t *codes = a.codes + (it.b * a.M + it.row0) * kb + (c0 >> 1);
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t *src = codes + (int64_t)(32 * i) * kb;
            q[i] = 0;
            if (it.row0 + 32 * i < a.M && FP8BQ_IN(FP4_SPAN_C(a), src, 4))
                asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(q[i]) : "l"(src));
        }
        const int tile = it.seg * (32 / TL) + lane / TL, blk = (lane % TL) / LPB;
        const uint8_t *run =
            a.scales + (it.tile_row * a.tiles_k + tile) * kFp4TileBytes + it.r * 16;
        uint4 sw = make_uint4(0u, 0u, 0u, 0u);
        if (FP8BQ_IN(FP4_SPAN_S(a), run, 16)) sw = __ldg((const uint4 *)run);
        const uint32_t sv[4] = {sw.x, sw.y, sw.z, sw.w};
        float t = 1.0f;
        if (FMT == FP8BQ_NVFP4 && a.tscale != nullptr &&
            FP8BQ_IN(FP4_SPAN_T(a), a.tscale + it.b * a.tbs, 4))
            t = __ldg(a.tscale + it.b * a.tbs);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (it.row0 + 32 * i >= a.M) break;
            const float s = scale_value<FMT>((sv[i] >> (8 * blk)) & 0xffu);
            float v[8];
            decode4(q[i], v[0], v[1], v[2], v[3]);
            decode4(q[i] >> 16, v[4], v[5], v[6], v[7]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = __fmul_rn(v[j], s);             // exact
                if (FMT == FP8BQ_NVFP4) v[j] = __fmul_rn(v[j], t);
            }
            char *dst = (char *)const_cast<void *>(a.x) +
                        (it.b * a.xbs + (int64_t)(it.row0 + 32 * i) * a.ld + c0) * OES;
            if constexpr (OES == 2) {
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[j]) : "f"(v[2 * j + 1]), "f"(v[2 * j]));
                if (VEC && n >= 8) {
                    if (FP8BQ_IN(FP4_SPAN_X(a), dst, 16))
                        asm volatile("st.global.cs.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(dst),
                                     "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]) : "memory");
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < n && FP8BQ_IN(FP4_SPAN_X(a), dst + 2 * j, 2))
                            *(uint16_t *)(dst + 2 * j) = (uint16_t)(o[j / 2] >> (16 * (j & 1)));
                }
            } else {
                if (VEC && n >= 8) {
                    if (FP8BQ_IN(FP4_SPAN_X(a), dst, 32))
                        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                                         dst),
                                     "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]),
                                     "f"(v[5]), "f"(v[6]), "f"(v[7])
                                     : "memory");
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < n && FP8BQ_IN(FP4_SPAN_X(a), dst + 4 * j, 4))
                            *(float *)(dst + 4 * j) = v[j];
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

template <int FMT, int ES, int MAXD>
cudaError_t quant_align(const Fp4Pack<MAXD> &p, int align, cudaStream_t st) {
    const unsigned grid = fp4_grid(p.total, 32);
    if (align >= 16) return launch_kernel(k_fp4_quant<FMT, ES, 16, MAXD>, grid, 256, 0, st, p);
    if (align >= 8) return launch_kernel(k_fp4_quant<FMT, ES, 8, MAXD>, grid, 256, 0, st, p);
    return launch_kernel(k_fp4_quant<FMT, ES, 1, MAXD>, grid, 256, 0, st, p);
}

template <int FMT, int OES, int MAXD>
cudaError_t dequant_vec(const Fp4Pack<MAXD> &p, bool vector, cudaStream_t st) {
    const unsigned grid = fp4_grid(p.total, 32);
    return vector ? launch_kernel(k_fp4_dequant<FMT, OES, true, MAXD>, grid, 256, 0, st, p)
                  : launch_kernel(k_fp4_dequant<FMT, OES, false, MAXD>, grid, 256, 0, st, p);
}

}  // namespace

template <int MAXD>
cudaError_t launch_fp4_quantize(const Fp4Pack<MAXD> &p, int format, int esize, int align,
                                cudaStream_t st) {
    if (format == FP8BQ_MXFP4)
        return esize == 2 ? quant_align<FP8BQ_MXFP4, 2>(p, align, st)
                          : quant_align<FP8BQ_MXFP4, 4>(p, align, st);
    return esize == 2 ? quant_align<FP8BQ_NVFP4, 2>(p, align, st)
                      : quant_align<FP8BQ_NVFP4, 4>(p, align, st);
}

template <int MAXD>
cudaError_t launch_fp4_dequantize(const Fp4Pack<MAXD> &p, int format, int esize, bool vector,
                                  cudaStream_t st) {
    if (format == FP8BQ_MXFP4)
        return esize == 2 ? dequant_vec<FP8BQ_MXFP4, 2>(p, vector, st)
                          : dequant_vec<FP8BQ_MXFP4, 4>(p, vector, st);
    return esize == 2 ? dequant_vec<FP8BQ_NVFP4, 2>(p, vector, st)
                      : dequant_vec<FP8BQ_NVFP4, 4>(p, vector, st);
}

template cudaError_t launch_fp4_quantize<kMaxDescSmall>(const Fp4Pack<kMaxDescSmall> &, int, int,
                                                        int, cudaStream_t);
template cudaError_t launch_fp4_quantize<kMaxFp4Large>(const Fp4Pack<kMaxFp4Large> &, int, int, int,
                                                       cudaStream_t);
template cudaError_t launch_fp4_dequantize<kMaxDescSmall>(const Fp4Pack<kMaxDescSmall> &, int, int,
                                                          bool, cudaStream_t);

FP8BQ_DEFINE_BOUNDS_RECORD(bounds_record_fp4_quant)

}  // namespace fp8bq
