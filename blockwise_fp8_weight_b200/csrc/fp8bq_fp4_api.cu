// fp8bq_fp4_api.cu -- the C ABI of the 4-bit operators: argument checks,
// grouping into launches, tensor maps of the products and the choice of their
// kernel.  A tensor map is made for each call from its arguments (under a
// microsecond each): nothing is kept from one call to the next.
#include <algorithm>
#include <atomic>
#include <cstring>
#include <vector>

#include "fp8bq_fp4.h"

using namespace fp8bq;

bool fp8bq::fp4_overlap(cudaStream_t st, double us) {
    if (!pdl_enabled()) return false;
    if (us >= pdl_min_us()) return true;
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &cs) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return cs != cudaStreamCaptureStatusNone;
}

namespace {

constexpr int64_t kMaxDim = (1ll << 31) - 256;
constexpr __int128 kMaxBytes = (__int128)1 << 62;

int esize_of(int32_t dtype) { return dtype == FP8BQ_BF16 ? 2 : 4; }
bool dtype_ok(int32_t d) { return d == FP8BQ_BF16 || d == FP8BQ_F32; }
bool format_ok(int32_t f) { return f == FP8BQ_MXFP4 || f == FP8BQ_NVFP4; }

// ------------------------------------------------------------------ overlap

struct Range {
    uintptr_t lo, hi;
    bool out;
};
void add_range(std::vector<Range> &v, const void *p, __int128 bytes, bool out) {
    if (p != nullptr && bytes > 0)
        v.push_back({(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, out});
}
// Outputs may overlap nothing; inputs may overlap each other.
bool overlaps(std::vector<Range> &v) {
    std::sort(v.begin(), v.end(), [](const Range &a, const Range &b) { return a.lo < b.lo; });
    uintptr_t out_end = 0, in_end = 0;
    for (const Range &r : v) {
        if (r.lo < out_end || (r.out && r.lo < in_end)) return true;
        (r.out ? out_end : in_end) = std::max(r.out ? out_end : in_end, r.hi);
    }
    return false;
}

// ------------------------------------------------------------------ quantise, dequantise

// One stack: `x` is the high-precision side (read or written).
struct Stack {
    const void *x;
    const uint8_t *codes, *scales;
    const float *tscale;
    int64_t M, K, ld, batch, xbs, tbs;
    int32_t dtype, format;

    int64_t code_bytes() const { return batch * M * fp4_row_bytes(K); }
    int64_t scale_bytes() const {
        return batch * fp4_tiles_m(M) * fp4_tiles_k(K, format) * kFp4TileBytes;
    }
    int64_t x_bytes() const { return ((batch - 1) * xbs + (M - 1) * ld + K) * esize_of(dtype); }
    int64_t t_bytes() const { return tscale ? ((batch - 1) * tbs + 1) * 4 : 0; }
};

fp8bq_status check_stack(Stack &D, bool x_is_output, bool *empty) {
    if (!dtype_ok(D.dtype)) return FP8BQ_ERR_DTYPE;
    if (!format_ok(D.format)) return FP8BQ_ERR_ARG;
    if (D.M < 0 || D.K < 0 || D.batch < 0 || D.ld < D.K || D.M > kMaxDim || D.K > kMaxDim)
        return FP8BQ_ERR_SHAPE;
    *empty = D.M == 0 || D.K == 0 || D.batch == 0;
    if (*empty) return FP8BQ_OK;
    if (D.batch == 1) D.xbs = D.tbs = 0;
    if (D.xbs < 0 || D.tbs < 0) return FP8BQ_ERR_SHAPE;
    if (D.x == nullptr || D.codes == nullptr || D.scales == nullptr) return FP8BQ_ERR_NULL;
    if (D.format == FP8BQ_MXFP4 && D.tscale != nullptr) return FP8BQ_ERR_ARG;
    const int es = esize_of(D.dtype);
    if ((uintptr_t)D.x % es || (uintptr_t)D.codes % 16 || (uintptr_t)D.scales % 16 ||
        (uintptr_t)D.tscale % 4)
        return FP8BQ_ERR_ALIGN;
    const __int128 b1 = D.batch - 1;
    if ((b1 * D.xbs + (__int128)(D.M - 1) * D.ld + D.K) * es > kMaxBytes ||
        (__int128)D.batch * D.M * fp4_row_bytes(D.K) > kMaxBytes ||
        (__int128)D.batch * fp4_tiles_m(D.M) * fp4_tiles_k(D.K, D.format) * kFp4TileBytes >
            kMaxBytes ||
        (b1 * D.tbs + 1) * 4 > kMaxBytes)
        return FP8BQ_ERR_SHAPE;
    if (x_is_output && D.batch > 1 && D.xbs < (D.M - 1) * D.ld + D.K) return FP8BQ_ERR_OVERLAP;
    return FP8BQ_OK;
}

void fill(const Stack &D, bool x_is_output, uint64_t begin, Fp4Desc *o) {
    o->x = D.x;
    o->codes = const_cast<uint8_t *>(D.codes);
    o->scales = const_cast<uint8_t *>(D.scales);
    o->tscale = D.tscale;
    o->ld = D.ld;
    o->xbs = D.xbs;
    o->tbs = D.tbs;
    o->M = (int32_t)D.M;
    o->K = (int32_t)D.K;
    o->tiles_m = (int32_t)fp4_tiles_m(D.M);
    o->tiles_k = (int32_t)fp4_tiles_k(D.K, D.format);
    o->begin = begin;
    const int64_t cols = fp4_item_cols(esize_of(D.dtype));
    o->items = (uint64_t)D.batch * fp4_tiles_m(D.M) * 32 * (uint64_t)((D.K + cols - 1) / cols);
#if FP8BQ_CHECKED
    o->x_bytes = x_is_output ? checked_extent(D.x_bytes()) : D.x_bytes();
    o->codes_bytes = x_is_output ? D.code_bytes() : checked_extent(D.code_bytes());
    o->scales_bytes = x_is_output ? D.scale_bytes() : checked_extent(D.scale_bytes());
    o->tscale_bytes = D.t_bytes();
#else
    (void)x_is_output;
#endif
}

// Bytes of the widest access that every row of the high-precision side allows.
int align_of(const Stack &D) {
    const int es = esize_of(D.dtype);
    for (int a : {32, 16, 8})
        if ((uintptr_t)D.x % a == 0 && (D.ld * es) % a == 0 && (D.xbs * es) % a == 0) return a;
    return es;
}

template <int MAXD>
cudaError_t quantize_group(const std::vector<Stack> &t, const std::vector<int> &idx, int align,
                           bool overlap, cudaStream_t st) {
    static thread_local Fp4Pack<MAXD> p;  // large: keep it off the stack
    const Stack &first = t[idx[0]];
    for (size_t i = 0; i < idx.size();) {
        p.n = p.pad_ = 0;
        p.total = 0;
        for (; i < idx.size() && p.n < MAXD; ++i, ++p.n) {
            fill(t[idx[i]], false, p.total, &p.d[p.n]);
            p.total += p.d[p.n].items;
        }
        const cudaError_t e =
            launch_fp4_quantize<MAXD>(p, first.format, esize_of(first.dtype), align, overlap, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

fp8bq_status run_quantize(std::vector<Stack> &t, cudaStream_t stream) {
    std::vector<Range> ranges;
    std::vector<int> groups[2][2][4];  // format, fp32 input, alignment
    static constexpr int kAligns[4] = {32, 16, 8, 0};
    bool any = false;
    double bytes = 0;
    for (size_t i = 0; i < t.size(); ++i) {
        bool empty = false;
        const fp8bq_status s = check_stack(t[i], false, &empty);
        if (s != FP8BQ_OK) return s;
        if (empty) continue;
        any = true;
        bytes += (double)t[i].batch * t[i].M * t[i].K * (esize_of(t[i].dtype) + 0.5);
        add_range(ranges, t[i].x, t[i].x_bytes(), false);
        add_range(ranges, t[i].codes, t[i].code_bytes(), true);
        add_range(ranges, t[i].scales, t[i].scale_bytes(), true);
        add_range(ranges, t[i].tscale, t[i].t_bytes(), false);
        const int a = align_of(t[i]);
        groups[t[i].format][t[i].dtype == FP8BQ_F32][a == 32 ? 0 : a == 16 ? 1 : a == 8 ? 2 : 3].push_back((int)i);
    }
    if (!any) return FP8BQ_OK;
    if (overlaps(ranges)) return FP8BQ_ERR_OVERLAP;
    const fp8bq_status sd = device_status();
    if (sd != FP8BQ_OK) return sd;
    const bool overlap = fp4_overlap(stream, 2 + bytes * 1.6e-7);
    for (auto &by_format : groups)
        for (auto &by_type : by_format)
            for (int a = 0; a < 4; ++a) {
                const std::vector<int> &g = by_type[a];
                if (g.empty()) continue;
                const cudaError_t e =
                    g.size() <= (size_t)kMaxDescSmall
                        ? quantize_group<kMaxDescSmall>(t, g, kAligns[a], overlap, stream)
                        : quantize_group<kMaxFp4Large>(t, g, kAligns[a], overlap, stream);
                if (e != cudaSuccess) {
                    cudaGetLastError();
                    return FP8BQ_ERR_DEVICE;
                }
            }
    return FP8BQ_OK;
}

Stack stack_of(const fp8bq_fp4_desc &D) {
    return {D.x,  D.codes, D.scales,         D.tensor_scale,        D.M,        D.K,
            D.ld, D.batch, D.x_batch_stride, D.tensor_scale_stride, D.dtype_in, D.format};
}

fp8bq_status run_dequantize(Stack D, cudaStream_t stream) {
    bool empty = false;
    const fp8bq_status s = check_stack(D, true, &empty);
    if (s != FP8BQ_OK || empty) return s;
    std::vector<Range> ranges;
    add_range(ranges, D.x, D.x_bytes(), true);
    add_range(ranges, D.codes, D.code_bytes(), false);
    add_range(ranges, D.scales, D.scale_bytes(), false);
    add_range(ranges, D.tscale, D.t_bytes(), false);
    if (overlaps(ranges)) return FP8BQ_ERR_OVERLAP;
    const fp8bq_status sd = device_status();
    if (sd != FP8BQ_OK) return sd;
    Fp4Pack<kMaxDescSmall> p;
    std::memset(&p, 0, sizeof p);
    p.n = 1;
    fill(D, true, 0, &p.d[0]);
    p.total = p.d[0].items;
    const int es = esize_of(D.dtype);
    const bool overlap =
        fp4_overlap(stream, 2 + (double)D.batch * D.M * D.K * (es + 0.5) * 1.6e-7);
    if (launch_fp4_dequantize<kMaxDescSmall>(p, D.format, es, align_of(D), overlap, stream) !=
        cudaSuccess) {
        cudaGetLastError();
        return FP8BQ_ERR_DEVICE;
    }
    return FP8BQ_OK;
}

// ------------------------------------------------------------------ products

struct Mat {
    const fp8bq_fp4_operand *o;
    int64_t rows, cbs, sbs, tbs;
    __int128 code_bytes, scale_bytes, t_bytes;
};

fp8bq_status check_operand(const fp8bq_fp4_operand &o, const fp8bq_fp4_matmul_desc &D, int64_t rows,
                           Mat *m) {
    if (o.codes == nullptr || o.scales == nullptr) return FP8BQ_ERR_NULL;
    if (D.format == FP8BQ_MXFP4 && o.tensor_scale != nullptr) return FP8BQ_ERR_ARG;
    const bool multi = D.batch > 1;
    m->o = &o;
    m->rows = rows;
    m->cbs = multi ? o.codes_batch_stride : 0;
    m->sbs = multi ? o.scales_batch_stride : 0;
    m->tbs = multi ? o.tensor_scale_stride : 0;
    if (m->cbs < 0 || m->sbs < 0 || m->tbs < 0) return FP8BQ_ERR_SHAPE;
    if ((uintptr_t)o.codes % 16 || (uintptr_t)o.scales % 16 || (uintptr_t)o.tensor_scale % 4 ||
        m->cbs % 16 || m->sbs % 16)
        return FP8BQ_ERR_ALIGN;
    const __int128 b1 = D.batch - 1;
    m->code_bytes = b1 * m->cbs + (__int128)rows * fp4_row_bytes(D.K);
    m->scale_bytes = b1 * m->sbs + (__int128)fp4_tiles_m(rows) * fp4_tiles_k(D.K, D.format) *
                                       kFp4TileBytes;
    m->t_bytes = o.tensor_scale ? (b1 * m->tbs + 1) * 4 : 0;
    // tensor maps take strides below 2^40 bytes
    if (m->code_bytes > kMaxBytes || m->scale_bytes > kMaxBytes || m->t_bytes > kMaxBytes ||
        m->cbs >= (1ll << 40) || m->sbs >= (1ll << 40))
        return FP8BQ_ERR_SHAPE;
    return FP8BQ_OK;
}

bool map_codes(const Mat &m, const fp8bq_fp4_matmul_desc &D, int box_rows, CUtensorMap *out) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const int64_t kb = fp4_row_bytes(D.K);
    const int64_t bs = m.cbs ? m.cbs : m.rows * kb < (1ll << 40) ? m.rows * kb : kb;
    cuuint64_t dims[3] = {(cuuint64_t)kb, (cuuint64_t)m.rows, (cuuint64_t)(m.cbs ? D.batch : 1)};
    cuuint64_t strides[2] = {(cuuint64_t)kb, (cuuint64_t)bs};
    cuuint32_t box[3] = {128, (cuuint32_t)box_rows, 1}, one[3] = {1, 1, 1};
    return fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(m.o->codes), dims,
              strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles as rows of 8-byte elements: one tile row of a stage (256
// columns) is one box.
bool map_scales(const Mat &m, const fp8bq_fp4_matmul_desc &D, CUtensorMap *out) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const int64_t row = fp4_tiles_k(D.K, D.format) * kFp4TileBytes, tm = fp4_tiles_m(m.rows);
    const int64_t bs = m.sbs ? m.sbs : tm * row < (1ll << 40) ? tm * row : row;
    cuuint64_t dims[3] = {(cuuint64_t)(row / 8), (cuuint64_t)tm, (cuuint64_t)(m.sbs ? D.batch : 1)};
    cuuint64_t strides[2] = {(cuuint64_t)row, (cuuint64_t)bs};
    cuuint32_t box[3] = {(cuuint32_t)(256 / (4 * fp4_block(D.format)) * kFp4TileBytes / 8), 1, 1};
    cuuint32_t one[3] = {1, 1, 1};
    return fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT64, 3, const_cast<uint8_t *>(m.o->scales), dims,
              strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A product that passed its checks, and how it is launched.
struct Product {
    Mat mats[3];
    __int128 out_bytes;
    int64_t obs, kb, stages;
    int store_align;
    int tokens;  // as from fp4_choose; -1: nothing to do
    double us;
};

std::atomic<int> g_force_tokens{-1};  // fp8bq_debug_set_fp4_tokens

// Whether tiles of that width (0: the many-token kernel) can compute M tokens.
bool tokens_ok(int tokens, int64_t M, bool gated) {
    return tokens == 0 || (tokens >= 64 ? tokens <= (gated ? 128 : 256) : M <= tokens);
}

fp8bq_status plan_product(const fp8bq_fp4_matmul_desc &D, bool gated, Product *P) {
    P->tokens = -1;
    if (!dtype_ok(D.dtype_out)) return FP8BQ_ERR_DTYPE;
    if (!format_ok(D.format)) return FP8BQ_ERR_ARG;
    if (D.M < 0 || D.N < 0 || D.batch < 0 || D.K < 1 || D.ld_out < D.N || D.M > kMaxDim ||
        D.N > kMaxDim || D.K > kMaxDim || D.batch > kMaxDim)
        return FP8BQ_ERR_SHAPE;
    if (D.M == 0 || D.N == 0 || D.batch == 0) return FP8BQ_OK;
    // the kernels number their tiles in 32 bits
    if (((__int128)(D.M + 15) / 16) * ((D.N + 127) / 128) * D.batch >= (1ll << 31))
        return FP8BQ_ERR_SHAPE;
    const int es = esize_of(D.dtype_out);
    const int64_t obs = P->obs = D.batch > 1 ? D.out_batch_stride : 0;
    if (obs < 0) return FP8BQ_ERR_SHAPE;
    if (D.out == nullptr) return FP8BQ_ERR_NULL;
    if ((uintptr_t)D.out % es || (uintptr_t)D.rows % 4) return FP8BQ_ERR_ALIGN;
    const __int128 out_bytes = P->out_bytes =
        ((__int128)(D.batch - 1) * obs + (__int128)(D.M - 1) * D.ld_out + D.N) * es;
    if (out_bytes > kMaxBytes) return FP8BQ_ERR_SHAPE;
    if (D.batch > 1 && obs < (D.M - 1) * D.ld_out + D.N) return FP8BQ_ERR_OVERLAP;
    Mat *mats = P->mats;
    const int n = gated ? 3 : 2;
    const uintptr_t out_lo = (uintptr_t)D.out, out_hi = out_lo + (uintptr_t)out_bytes;
    auto in_out = [&](const void *q, __int128 bytes) {
        return q != nullptr && bytes > 0 && (uintptr_t)q < out_hi &&
               out_lo < (uintptr_t)q + (uintptr_t)bytes;
    };
    bool overlap = in_out(D.rows, (__int128)D.batch * 4);
    for (int i = 0; i < n; ++i) {
        const fp8bq_fp4_operand &o = i == 0 ? D.a : i == 1 ? D.b : D.up;
        const fp8bq_status s = check_operand(o, D, i == 0 ? D.M : D.N, &mats[i]);
        if (s != FP8BQ_OK) return s;
        overlap |= in_out(o.codes, mats[i].code_bytes) || in_out(o.scales, mats[i].scale_bytes) ||
                   in_out(o.tensor_scale, mats[i].t_bytes);
    }
    if (overlap) return FP8BQ_ERR_OVERLAP;
    P->kb = fp4_row_bytes(D.K);
    P->stages = (P->kb + 127) / 128;
    P->store_align = es;
    for (int a : {4, 8, 16, 32})
        if ((uintptr_t)D.out % a == 0 && D.ld_out * es % a == 0 && obs * es % a == 0)
            P->store_align = a;
    P->tokens = fp4_choose(D.M, D.N, P->stages, D.batch, gated, fp4_staged(P->store_align, es), &P->us);
    const int force = g_force_tokens.load(std::memory_order_relaxed);
    if (force >= 0 && tokens_ok(force, D.M, gated)) P->tokens = force;
    return FP8BQ_OK;
}

fp8bq_status run_matmul(const fp8bq_fp4_matmul_desc *desc, bool gated, cudaStream_t stream) {
    if (desc == nullptr) return FP8BQ_ERR_NULL;
    const fp8bq_fp4_matmul_desc &D = *desc;
    Product P;
    const fp8bq_status s = plan_product(D, gated, &P);
    if (s != FP8BQ_OK || P.tokens < 0) return s;
    const fp8bq_status sd = device_status();
    if (sd != FP8BQ_OK) return sd;
    const Mat *mats = P.mats;
    const int n = gated ? 3 : 2;
    const bool wide = P.tokens == 0;
    Fp4MmParams p;
    std::memset(&p, 0, sizeof p);
    bool ok = map_codes(mats[0], D, wide ? 128 : P.tokens, &p.x) && map_scales(mats[0], D, &p.xs);
    for (int i = 1; ok && i < n; ++i)
        ok = map_codes(mats[i], D, 128, &p.w[i - 1]) && map_scales(mats[i], D, &p.ws[i - 1]);
    if (!ok) return FP8BQ_ERR_DEVICE;
    p.xt = D.a.tensor_scale;
    p.xtbs = mats[0].tbs;
    for (int i = 1; i < n; ++i) {
        p.wt[i - 1] = mats[i].o->tensor_scale;
        p.wtbs[i - 1] = mats[i].tbs;
    }
    p.out = D.out;
    p.rows = D.rows;
    p.ldo = D.ld_out;
    p.obs = P.obs;
    p.wait_limit_ns = wait_limit();
    p.M = (int32_t)D.M;
    p.N = (int32_t)D.N;
    p.batch = (int32_t)D.batch;
    p.stages_k = (int32_t)P.stages;
    p.mma_k = (int32_t)((P.kb + 31) / 32);
    p.split = 1;
    p.store_align = P.store_align;
    for (int i = 0; i < n; ++i)  // a stack stride of 0: one matrix for the whole stack
        p.moves |= (mats[i].cbs ? 1u : 0u) << (2 * i) | (mats[i].sbs ? 2u : 0u) << (2 * i);
    p.overlap = fp4_overlap(stream, P.us);
    p.inject = inject_flags();
#if FP8BQ_CHECKED
    p.out_bytes = checked_extent((uint64_t)P.out_bytes);
    p.rows_bytes = (uint64_t)D.batch * 4;
    p.xt_bytes = (uint64_t)mats[0].t_bytes;
    for (int i = 1; i < n; ++i) p.wt_bytes[i - 1] = (uint64_t)mats[i].t_bytes;
#endif
    const bool bf16 = D.dtype_out == FP8BQ_BF16;
    if ((wide ? launch_fp4_mm_wide(p, D.format, gated, bf16, stream)
              : launch_fp4_mm_narrow(p, D.format, gated, bf16, P.tokens, stream)) != cudaSuccess) {
        cudaGetLastError();
        return FP8BQ_ERR_DEVICE;
    }
    return FP8BQ_OK;
}

// No C++ exception leaves an entry point: the lists above are the only
// allocations, and a host without memory for them is reported as such.
template <typename F>
fp8bq_status guarded(F &&f) {
    try {
        return f();
    } catch (...) {
        return FP8BQ_ERR_DEVICE;
    }
}

}  // namespace

extern "C" {

fp8bq_status fp8bq_fp4_quantize(const void *x, fp8bq_dtype dtype_in, int64_t M, int64_t K,
                                int64_t ld, fp8bq_fp4_format format, const float *tensor_scale,
                                uint8_t *codes, uint8_t *scales, cudaStream_t stream) {
    return guarded([&] {
        std::vector<Stack> t{{x, codes, scales, tensor_scale, M, K, ld, 1, 0, 0, (int32_t)dtype_in,
                              (int32_t)format}};
        return run_quantize(t, stream);
    });
}

fp8bq_status fp8bq_fp4_quantize_batched(const fp8bq_fp4_desc *desc_table, int n_tensors,
                                        cudaStream_t stream) {
    if (n_tensors < 0) return FP8BQ_ERR_ARG;
    if (n_tensors > 0 && desc_table == nullptr) return FP8BQ_ERR_NULL;
    return guarded([&] {
        std::vector<Stack> t;
        t.reserve((size_t)n_tensors);
        for (int i = 0; i < n_tensors; ++i) t.push_back(stack_of(desc_table[i]));
        return run_quantize(t, stream);
    });
}

fp8bq_status fp8bq_fp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t batch,
                                  int64_t M, int64_t K, fp8bq_fp4_format format,
                                  const float *tensor_scale, int64_t tensor_scale_stride, void *out,
                                  fp8bq_dtype dtype_out, int64_t ld_out, int64_t out_batch_stride,
                                  cudaStream_t stream) {
    return guarded([&] {
        return run_dequantize({out, codes, scales, tensor_scale, M, K, ld_out, batch,
                               out_batch_stride, tensor_scale_stride, (int32_t)dtype_out,
                               (int32_t)format},
                              stream);
    });
}

fp8bq_status fp8bq_debug_set_fp4_tokens(int tokens) {
    for (int t : {-1, 0, 16, 32, 64, 128, 256})
        if (t == tokens) {
            g_force_tokens.store(tokens);
            return FP8BQ_OK;
        }
    return FP8BQ_ERR_ARG;
}

fp8bq_status fp8bq_fp4_plan(const fp8bq_fp4_matmul_desc *desc, int gated, int *tokens, int *overlap) {
    if (desc == nullptr) return FP8BQ_ERR_NULL;
    Product P;
    const fp8bq_status s = plan_product(*desc, gated != 0, &P);
    if (s != FP8BQ_OK) return s;
    if (tokens) *tokens = P.tokens;
    if (overlap) *overlap = P.tokens < 0 ? -1 : pdl_enabled() && P.us >= pdl_min_us();
    return FP8BQ_OK;
}

fp8bq_status fp8bq_fp4_matmul(const fp8bq_fp4_matmul_desc *desc, cudaStream_t stream) {
    return guarded([&] { return run_matmul(desc, false, stream); });
}

fp8bq_status fp8bq_fp4_gated_matmul(const fp8bq_fp4_matmul_desc *desc, cudaStream_t stream) {
    return guarded([&] { return run_matmul(desc, true, stream); });
}

}  // extern "C"
