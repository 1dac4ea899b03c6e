// fp8bq_fp4.h -- what the host side of the 4-bit operators (quantise,
// dequantise, product, gated product) and their kernels share.
#pragma once

#include <cudaTypedefs.h>  // PFN_cuTensorMapEncodeTiled

#include "../../include/fp8bq.h"
#include "fp8bq_internal.h"

namespace fp8bq {

// Process-wide state of the library that the 4-bit entry points use too
// (fp8bq_api.cu).
fp8bq_status device_status();       // FP8BQ_OK if the current device is usable
uint64_t wait_limit();              // bound of a device wait, ns
uint32_t inject_flags();            // FP8BQ_INJECT_*
uint64_t checked_extent(uint64_t);  // an output's extent for the bounds checks
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Whether a call that takes the device about `us` microseconds is launched
// with programmatic stream serialization: if it is on, unless the call is
// shorter than pdl_min_us() and outside a graph.  The attribute costs the host
// 1.6 us a launch (4.2 against 2.6 measured) and saves the device 2 to 3, so a
// caller who needs longer for a call than the device does gains by leaving it
// out.  (515 tokens against 1000 x 4100, about 8 us, through the Python binding:
// 12.3 us a call without it, 9.6 with; one token against 6144 x 4096 in a loop of
// C calls: 8.9 without, 6.5 with.)
double pdl_min_us();                // fp8bq_set_pdl_min_us
bool fp4_overlap(cudaStream_t st, double us);

// ------------------------------------------------------------------ layout
//
// Codes: rows of 16 * ceil(K / 32) bytes.  Scales: tiles of 128 rows by four
// blocks, 512 bytes each: the order in which the tensor cores take them from
// shared memory, so a tile goes there as it lies in memory.
constexpr int kFp4TileRows = 128;
constexpr int kFp4TileBytes = 512;
constexpr int fp4_block(int format) { return format == FP8BQ_MXFP4 ? 32 : 16; }
inline int64_t fp4_row_bytes(int64_t K) { return (K + 31) / 32 * 16; }
inline int64_t fp4_tiles_m(int64_t M) { return (M + kFp4TileRows - 1) / kFp4TileRows; }
inline int64_t fp4_tiles_k(int64_t K, int format) {
    const int64_t w = 4 * fp4_block(format);
    return (K + w - 1) / w;
}

// ------------------------------------------------------------------ quantise, dequantise
//
// A work item is a warp's: rows r, r + 32, r + 64 and r + 96 of a 128-row
// tile row by a run of columns, so that the scales of an item fill whole
// 16-byte runs of the tiles.  The run: 32 bytes a lane of the high-precision
// side.
constexpr int fp4_item_cols(int esize) { return 32 * (32 / esize); }

struct Fp4Desc {
    const void *x;       // high-precision side: input, or output of dequantise
    uint8_t *codes, *scales;
    const float *tscale; // the tensor's own scale, or NULL (1)
    int64_t ld, xbs;     // elements
    int64_t tbs;         // floats between the stacks' tensor scales (0 or 1)
    int32_t M, K;
    int32_t tiles_m, tiles_k;
    uint64_t begin, items;
#if FP8BQ_CHECKED
    uint64_t x_bytes, codes_bytes, scales_bytes, tscale_bytes;
#endif
};

template <int MAXD>
struct Fp4Pack {
    int32_t n;
    int32_t pad_;
    uint64_t total;
    Fp4Desc d[MAXD];
};
constexpr int kMaxFp4Large = FP8BQ_CHECKED ? 224 : 288;
static_assert(sizeof(Fp4Pack<kMaxFp4Large>) < 32000, "kernel parameter limit");

// align: bytes of the widest access every row of the high-precision side
// allows (32, 16, 8 or the element's size)
template <int MAXD>
cudaError_t launch_fp4_quantize(const Fp4Pack<MAXD> &p, int format, int esize, int align,
                                bool overlap, cudaStream_t st);
template <int MAXD>
cudaError_t launch_fp4_dequantize(const Fp4Pack<MAXD> &p, int format, int esize, int align,
                                  bool overlap, cudaStream_t st);

// ------------------------------------------------------------------ products

struct Fp4MmParams {
    CUtensorMap x, w[2];    // codes: tokens, weight (gated: gate and up)
    CUtensorMap xs, ws[2];  // their scales
    const float *xt, *wt[2];
    int64_t xtbs, wtbs[2];
    void *out;
    const int32_t *rows;  // valid rows of each matrix of the stack, or NULL
    int64_t ldo, obs;
    uint64_t wait_limit_ns;
    int32_t M, N, batch;
    int32_t stages_k;  // ceil(K / 256)
    int32_t mma_k;     // ceil(K / 64)
    int32_t overlap;   // launch with programmatic stream serialization (host)
    int32_t split;     // CTAs that share a tile's K range (a cluster)
    int32_t store_align; // bytes (32, 16, 8 or the element's) that every output row is aligned to
    uint32_t moves;    // bit i: operand map i steps with the stack (x, xs, w[0], ws[0], w[1], ws[1])
    uint32_t inject;
#if FP8BQ_CHECKED
    uint64_t out_bytes, rows_bytes, xt_bytes, wt_bytes[2];
#endif
};

// tokens: the tile's width in tokens (16, 32, 64, 128 or 256; gated at most 128)
cudaError_t launch_fp4_mm_narrow(const Fp4MmParams &p, int format, bool gated, bool out_bf16,
                                 int tokens, cudaStream_t st);
// Whether the many-token kernel's outputs pass through shared memory.
constexpr bool fp4_staged(int store_align, int esize) { return store_align < 8 * esize; }
// Which kernel: 0 the one for many tokens, else the tile's width in tokens; `us`:
// the microseconds it takes about.
int fp4_choose(int64_t M, int64_t N, int64_t stages, int64_t batch, bool gated, bool staged,
               double *us);
// Tiles of 256 tokens by 256 outputs (gated: 128) on pairs of SMs.
cudaError_t launch_fp4_mm_wide(const Fp4MmParams &p, int format, bool gated, bool out_bf16,
                               cudaStream_t st);

cudaError_t read_and_clear_fp4_error_word(uint32_t *out);
cudaError_t bounds_record_fp4_quant(uint64_t *count, uint64_t *first, bool clear);
cudaError_t bounds_record_fp4_mm(uint64_t *count, uint64_t *first, bool clear);

}  // namespace fp8bq
