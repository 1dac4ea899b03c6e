// fp8bq_fp4_mm.cu -- products of 4-bit matrices on the block-scaled tensor
// cores: out = a b^T, and out = silu(a b^T) * (a up^T).
//
// The codes go from memory to shared memory as they are (TMA, 128-byte
// swizzle: 256 codes of a row), the scale tiles too; a scale tile is copied
// into tensor memory next to the fp32 sums, and tcgen05.mma multiplies codes
// and scales of 64 columns of K at a time.  Nothing is unpacked.
#include "fp8bq_fp4_device.cuh"

namespace fp8bq {

// Bits as in the TMA quantiser's error word: 1 a wait ran out, 2 a copy or a
// product may still be in flight.
__device__ uint32_t g_fp4_error_word;

namespace {

constexpr uint64_t kDrainNs = 2000000000ull;

#define MM_SPAN(base, bytes) (dev::Span{(uint64_t)(base), (uint64_t)(base) + (bytes)})

// v / (1 + exp(-v)) by the fast exponential and division: their documented
// errors are 2 + |1.173 v| and 2 units in the last place, far below the
// rounding of a bf16 output and of the order of an fp32 sum's own.  (expf and
// the IEEE division: 313 us instead of 62 for 8192 x 6144 outputs over
// K = 512, on B200.)
__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.0f + __expf(-v)); }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// A tensor's own scale for matrix e.
__device__ __forceinline__ float tensor_scale(const float *t, int64_t stride, int64_t e,
                                              [[maybe_unused]] uint64_t bytes) {
    if (t == nullptr || !FP8BQ_IN(MM_SPAN(t, bytes), t + e * stride, 4)) return 1.0f;
    return __ldg(t + e * stride);
}
#if FP8BQ_CHECKED
#define MM_XT(p, e) tensor_scale((p).xt, (p).xtbs, e, (p).xt_bytes)
#define MM_WT(p, i, e) tensor_scale((p).wt[i], (p).wtbs[i], e, (p).wt_bytes[i])
#else
#define MM_XT(p, e) tensor_scale((p).xt, (p).xtbs, e, 0)
#define MM_WT(p, i, e) tensor_scale((p).wt[i], (p).wtbs[i], e, 0)
#endif

// Valid rows of matrix e.
__device__ __forceinline__ int valid_rows(const Fp4MmParams &p, int e) {
    if (p.rows == nullptr || !FP8BQ_IN(MM_SPAN(p.rows, p.rows_bytes), p.rows + e, 4)) return p.M;
    return max(0, min(p.M, *(p.rows + e)));
}

// Four consecutive outputs of row m from column n (n a multiple of 4).
template <bool BF16>
__device__ __forceinline__ void store4(const Fp4MmParams &p, int64_t e, int64_t m, int n,
                                       const float (&v)[4]) {
    constexpr int ES = BF16 ? 2 : 4;
    char *dst = (char *)p.out + (e * p.obs + m * p.ldo + n) * ES;
    if (p.store_align >= 4 * ES && n + 4 <= p.N) {
        if (!FP8BQ_IN(MM_SPAN(p.out, p.out_bytes), dst, 4 * ES)) return;
        if constexpr (BF16) *(uint2 *)dst = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
        else *(float4 *)dst = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < p.N && FP8BQ_IN(MM_SPAN(p.out, p.out_bytes), dst + j * ES, ES)) {
                if constexpr (BF16) *(uint16_t *)(dst + j * ES) = (uint16_t)bf16x2(v[j], 0.0f);
                else *(float *)(dst + j * ES) = v[j];
            }
    }
}

// ============================================================== few tokens
//
// A CTA computes 128 outputs (rows of the weight, the M side of the tensor
// core's tile) for NT tokens (its N side): few tokens cost few MMA columns,
// and the kernel is bound by the weight's bytes.  Where the tiles are too few
// to keep every SM loading, a cluster of `split` CTAs shares a tile: each sums
// a run of K, the partial sums meet in shared memory, and every CTA of the
// cluster adds up and stores a part of the tile, in the order of the ranks:
// no atomics, no workspace, the same sum every time.
//
// Warp 0 loads (one lane), warp 1 issues the products (one lane), all four
// warps store.  Every wait is bounded; one that runs out sets the error word,
// and the CTA still waits for its copies and products before it leaves.
template <int FMT, bool GATED, int NT>
struct Narrow {
    static constexpr int W = GATED ? 2 : 1;
    static constexpr int KT = 256 / (4 * fp4_block(FMT));   // scale tiles along a stage's K
    static constexpr int SF = KT * kFp4TileBytes;           // scales of 128 rows
    static constexpr int XT = (NT + 127) / 128;             // token scale tile rows
    static constexpr int kCodesW = 128 * 128;
    static constexpr int kCodesX = NT * 128;
    static constexpr int kStage = W * (kCodesW + SF) + kCodesX + XT * SF;
    // two buffers of scale columns after the sums
    static constexpr int kSfCols = 4 * KT * (W + XT);
    static constexpr int kNeed = W * NT + 2 * kSfCols;
    static constexpr int kCols = kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
    static_assert(kNeed <= 512, "tensor memory");
    // Two CTAs an SM where the sums leave room, else one.  A CTA that takes
    // c of the 512 tensor-memory columns takes at least c / 512 of the SM's
    // shared memory, so CTAs that share an SM always find their columns and
    // none waits for another's while a third waits for it.
    static constexpr int kSmall = 114688, kLarge = 231424;  // 112 KB, 226 KB
    static constexpr int kSmem = kCols <= 128 || (kCols == 256 && 2 * kStage + 1024 <= kSmall)
                                     ? kSmall
                                     : kLarge;
    static constexpr int kStages = (kSmem - 1024) / kStage;
    static_assert(kStages >= 2, "ring");
    static_assert(W * NT * 128 * 4 <= kStages * kStage, "partial sums");
};

template <int FMT, bool GATED, bool BF16, int NT>
__global__ void __launch_bounds__(128) k_fp4_narrow(const __grid_constant__ Fp4MmParams p) {
    using S = Narrow<FMT, GATED, NT>;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages], sums;
    __shared__ uint32_t tmem_at;
    __shared__ volatile int abort_flag;
    uint8_t *ring = raw + ((1024u - (dev::smem_addr(raw) & 1023u)) & 1023u);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)(blockIdx.x % (unsigned)p.split);
    const int n0 = (int)(blockIdx.x / (unsigned)p.split) * 128;
    const int m0 = (int)blockIdx.y * NT;
    const int e = (int)blockIdx.z;
    if (tid == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            dev::mbar_init(&full[s], 1);
            dev::mbar_init(&empty[s], 1);
        }
        dev::mbar_init(&sums, 1);
        abort_flag = 0;
        dev::fence_mbar_init();
        dev::prefetch_tensormap(&p.w[0]);
        dev::prefetch_tensormap(&p.x);
    }
    if (warp == 1) dev::tmem_alloc<1>(&tmem_at, S::kCols);
    dev::tc_fence_before();
    __syncthreads();
    dev::tc_fence_after();
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    const uint32_t tmem = tmem_at;
    const int valid = min(NT, valid_rows(p, e) - m0);
    if (valid > 0) {  // the same for every CTA of a cluster
        const int k0 = (int)((int64_t)p.stages_k * rank / p.split);
        const int k1 = (int)((int64_t)p.stages_k * (rank + 1) / p.split);
        if (warp == 0 && lane == 0) {
            bool dropped = false;
            auto at = [&](int map) { return (p.moves >> map) & 1u ? e : 0; };
            int i = 0;
            for (; k0 + i < k1; ++i) {
                const int st = i % S::kStages, round = i / S::kStages, k = k0 + i;
                if (round > 0 && !dev::mbar_wait_bounded(&empty[st], (round - 1) & 1,
                                                         p.wait_limit_ns, &abort_flag)) {
                    if (!abort_flag) {
                        atomicOr(&g_fp4_error_word, 1u);
                        abort_flag = 1;
                    }
                    break;
                }
                dev::mbar_arrive_expect_tx(&full[st], S::kStage);
                if ((p.inject & FP8BQ_INJECT_DROP_FIRST_LOAD) && i == 0 &&
                    (blockIdx.x | blockIdx.y | blockIdx.z) == 0) {
                    dropped = true;
                    continue;
                }
                uint8_t *b = ring + st * S::kStage;
#pragma unroll
                for (int w = 0; w < S::W; ++w, b += S::kCodesW)
                    dev::tma_load_3d(b, &p.w[w], &full[st], k * 128, n0, at(2 + 2 * w), false);
                dev::tma_load_3d(b, &p.x, &full[st], k * 128, m0, at(0), false);
                b += S::kCodesX;
#pragma unroll
                for (int w = 0; w < S::W; ++w, b += S::SF)
                    dev::tma_load_3d(b, &p.ws[w], &full[st], k * (S::SF / 8), n0 / 128, at(3 + 2 * w),
                                     false);
#pragma unroll
                for (int t = 0; t < S::XT; ++t, b += S::SF)
                    dev::tma_load_3d(b, &p.xs, &full[st], k * (S::SF / 8), m0 / 128 + t, at(1), false);
            }
            for (int st = 0; st < S::kStages && st < i; ++st) {  // every copy has landed
                const int fills = (i - st + S::kStages - 1) / S::kStages;
                if (dropped && st == 0 && fills == 1) continue;
                if (!dev::mbar_wait_bounded(&full[st], (fills - 1) & 1, kDrainNs, nullptr))
                    atomicOr(&g_fp4_error_word, 2u);
            }
        } else if (warp == 1 && lane == 0) {
            constexpr uint32_t word = dev::mma_word(FMT, 128, NT);
            for (int i = 0; k0 + i < k1; ++i) {
                const int st = i % S::kStages, k = k0 + i;
                if (!dev::mbar_wait_bounded(&full[st], (i / S::kStages) & 1, p.wait_limit_ns,
                                            &abort_flag)) {
                    if (!abort_flag) {
                        atomicOr(&g_fp4_error_word, 1u);
                        abort_flag = 1;
                    }
                    break;
                }
                dev::tc_fence_after();
                const uint32_t at = dev::smem_addr(ring + st * S::kStage);
                const uint32_t sf = at + S::W * S::kCodesW + S::kCodesX;
                const uint32_t sw = tmem + S::W * NT + (i & 1) * S::kSfCols;
                const uint32_t sx = sw + 4 * S::KT * S::W;
#pragma unroll
                for (int t = 0; t < S::KT; ++t) {
#pragma unroll
                    for (int w = 0; w < S::W; ++w)
                        dev::scales_to_tmem<1>(sw + 4 * (w * S::KT + t),
                                               dev::scale_desc(sf + w * S::SF + t * kFp4TileBytes));
#pragma unroll
                    for (int x = 0; x < S::XT; ++x)
                        dev::scales_to_tmem<1>(
                            sx + 4 * (t * S::XT + x),
                            dev::scale_desc(sf + (S::W + x) * S::SF + t * kFp4TileBytes));
                }
                const uint64_t xd = dev::operand_desc(at + S::W * S::kCodesW);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (4 * k + j >= p.mma_k) break;
                    const int t = j * S::KT / 4;
                    const uint32_t wd = dev::mma_word_id(word, FMT == FP8BQ_MXFP4 ? 2 * (j & 1) : 0);
#pragma unroll
                    for (int w = 0; w < S::W; ++w)
                        dev::mma_fp4<FMT, 1>(tmem + w * NT,
                                             dev::operand_desc(at + w * S::kCodesW) + 2 * j,
                                             xd + 2 * j, wd, sw + 4 * (w * S::KT + t),
                                             sx + 4 * t * S::XT, i + j > 0);
                }
                dev::mma_commit<1>(&empty[st]);
            }
            dev::mma_commit<1>(&sums);
        }
        __syncwarp();
        // The products give up on their own; a little longer, and they are stuck.
        bool ok = dev::mbar_wait_bounded(&sums, 0, 2 * p.wait_limit_ns + kDrainNs, nullptr);
        if (!ok && tid == 0) atomicOr(&g_fp4_error_word, 2u);
        dev::tc_fence_after();
        // Sums to shared memory (the ring is free: every copy was waited for
        // and every product is done), [weight][token][128 outputs].
        float *part = reinterpret_cast<float *>(ring);
#pragma unroll
        for (int w = 0; w < S::W; ++w) {
#pragma unroll
            for (int c = 0; c < NT; c += 16) {
                if (c >= valid) break;
                uint32_t v[16];
                dev::tmem_ld16(tmem + ((uint32_t)(warp * 32) << 16) + w * NT + c, v);
                dev::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    part[(w * NT + c + j) * 128 + tid] = __uint_as_float(v[j]);
            }
        }
        dev::tc_fence_before();
        if (p.split > 1) dev::cluster_sync();
        else __syncthreads();
        ok = ok && !abort_flag;
        const float xt = MM_XT(p, e);
        float alpha[S::W];
#pragma unroll
        for (int w = 0; w < S::W; ++w) alpha[w] = __fmul_rn(xt, MM_WT(p, w, e));
        const uint32_t at = dev::smem_addr(part);
        for (int q = rank * 128 + tid; ok && q < valid * 32; q += p.split * 128) {
            const int t = q >> 5, n = n0 + (q & 31) * 4;
            if (n >= p.N) continue;
            float v[S::W][4];
#pragma unroll
            for (int w = 0; w < S::W; ++w) {
                const uint32_t a = at + ((w * NT + t) * 128 + (q & 31) * 4) * 4;
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int r = 0; r < p.split; ++r) {
                    const float4 o = p.split > 1
                                         ? dev::peer_ld4(dev::peer_addr(a, r))
                                         : *reinterpret_cast<const float4 *>(
                                               part + (w * NT + t) * 128 + (q & 31) * 4);
                    s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
                }
                v[w][0] = s.x * alpha[w], v[w][1] = s.y * alpha[w];
                v[w][2] = s.z * alpha[w], v[w][3] = s.w * alpha[w];
            }
            if constexpr (GATED)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[0][j] = silu(v[0][j]) * v[S::W - 1][j];
            store4<BF16>(p, e, m0 + t, n, v[0]);
        }
        if (p.split > 1) dev::cluster_sync();  // peers may still read this CTA's sums
    }
    __syncthreads();
    if (warp == 1) dev::tmem_dealloc<1>(tmem, S::kCols);
}

// ============================================================== many tokens
//
// A pair of SMs (cta_group::2) computes 256 tokens by 256 outputs: each CTA
// holds the codes of its 128 tokens and of half of the weight's 256 rows, and
// the tensor cores of both read both halves, so a stage of 256 columns of K
// costs each SM 32 KB of codes for 128 x 256 outputs.  Gated: 128 outputs, the
// first half of the 256 weight rows from the gate, the other from `up`, so the
// two sums of an output lie 128 columns apart in the same tensor-memory lane.
//
// Persistent: a pair walks over tiles.  In each CTA warp 0 loads (one lane),
// warps 4-7 bring the scales into tensor memory, warps 8-15 store; warp 1 of
// the first CTA issues the products of both.  The sums of successive tiles
// alternate between columns [0, 256) and [160, 416), so the next tile is
// multiplied while this one is stored; the 96 columns that both use are stored
// first, and the next tile waits for those alone.  The scales' buffers take
// the last 96 columns.
//
// The scales go through registers (ld.shared, tcgen05.st) rather than by
// tcgen05.cp: a copy of one scale tile holds up the tensor cores for 62
// clocks, and a stage has 6 (mxfp4) or 12 (nvfp4) of them beside 768 clocks of
// products.  Measured on B200, 8192 tokens against 6144 x 16384: clocks a
// stage 1240 / 1570 with the copies.
template <int FMT>
struct Wide {
    static constexpr int KT = 256 / (4 * fp4_block(FMT));
    static constexpr int SF = KT * kFp4TileBytes;
    static constexpr int kCodes = 128 * 128;                   // 128 rows
    static constexpr int kStage = 2 * kCodes + 3 * SF;         // tokens, weight, their scales
    static constexpr int kSmem = 231424;                       // an SM to itself
    static constexpr int kStages = (kSmem - 1024) / kStage;
    static constexpr int kOther = 160;                         // columns of the odd tiles' sums
    static constexpr int kScales = 416;
    static constexpr int kSfCols = 12 * KT;                    // a stage's: tokens, then weight
    static constexpr int kSfBufs = (512 - kScales) / kSfCols;
    static constexpr int kThreads = 512;
    static_assert(kSfBufs >= 2 && kSfBufs <= kStages, "scale buffers");
};

// 32 consecutive outputs of a row, from column n; `align` bytes.
template <bool BF16>
__device__ __forceinline__ void store32(const Fp4MmParams &p, int64_t e, int64_t m, int n,
                                        const float (&v)[32]) {
    constexpr int ES = BF16 ? 2 : 4, PER = 32 / ES;            // outputs in 32 bytes
    char *dst = (char *)p.out + (e * p.obs + m * p.ldo + n) * ES;
#pragma unroll
    for (int c = 0; c < 32; c += PER, dst += 32) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = BF16 ? bf16x2(v[(c + 2 * j) & 31], v[(c + 2 * j + 1) & 31])
                        : __float_as_uint(v[(c + j) & 31]);
        if (n + c + PER <= p.N && p.store_align >= 16) {
            if (!FP8BQ_IN(MM_SPAN(p.out, p.out_bytes), dst, 32)) continue;
            if (p.store_align >= 32) {
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst),
                             "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]),
                             "r"(w[6]), "r"(w[7])
                             : "memory");
            } else {
                *(uint4 *)dst = make_uint4(w[0], w[1], w[2], w[3]);
                *(uint4 *)(dst + 16) = make_uint4(w[4], w[5], w[6], w[7]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (n + c + j < p.N &&
                    FP8BQ_IN(MM_SPAN(p.out, p.out_bytes), dst + j * ES, ES)) {
                    if constexpr (BF16)
                        *(uint16_t *)(dst + j * 2) = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
                    else
                        *(uint32_t *)(dst + j * 4) = w[j & 7];
                }
        }
    }
}

// The tiles of a pair: first rows, first outputs and matrix of the stack, in
// the same order for every role; tiles without valid rows are passed over.
struct WideWalk {
    const Fp4MmParams &p;
    int64_t t, step, total;
    int mt, nt, width;
    int m0, n0, e, valid;
    __device__ __forceinline__ WideWalk(const Fp4MmParams &q, int width_)
        : p(q), t((int64_t)(blockIdx.x >> 1) - (gridDim.x >> 1)), step(gridDim.x >> 1), width(width_) {
        mt = (p.M + 255) / 256;
        nt = (p.N + width - 1) / width;
        total = (int64_t)mt * nt * p.batch;
    }
    __device__ __forceinline__ bool next() {
        while ((t += step) < total) {
            const int64_t r = t / mt;
            e = (int)(r / nt);
            m0 = (int)(t - r * mt) * 256;
            n0 = (int)(r - (int64_t)e * nt) * width;
            valid = valid_rows(p, e);
            if (m0 < valid) return true;
        }
        return false;
    }
};

template <int FMT, bool GATED, bool BF16>
__global__ void __launch_bounds__(512, 1) k_fp4_wide(const __grid_constant__ Fp4MmParams p) {
    using S = Wide<FMT>;
    extern __shared__ uint8_t raw[];
    // full (codes), scaled, drained: the first CTA's count for both; landed
    // (scales), empty, sums: each CTA its own
    __shared__ __align__(8) uint64_t full[S::kStages], landed[S::kStages], empty[S::kStages];
    __shared__ __align__(8) uint64_t scaled[S::kSfBufs], sums, drained, done;
    __shared__ uint32_t tmem_at;
    __shared__ volatile int abort_flag;
    uint8_t *ring = raw + ((1024u - (dev::smem_addr(raw) & 1023u)) & 1023u);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = dev::cluster_rank();
    constexpr int kWidth = GATED ? 128 : 256;
    if (tid == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            dev::mbar_init(&full[s], 1);
            dev::mbar_init(&landed[s], 1);
            dev::mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < S::kSfBufs; ++s) dev::mbar_init(&scaled[s], 8);
        dev::mbar_init(&sums, 1);
        dev::mbar_init(&drained, 16);
        dev::mbar_init(&done, 1);
        abort_flag = 0;
        dev::fence_mbar_init();
        dev::prefetch_tensormap(&p.w[0]);
        dev::prefetch_tensormap(&p.x);
    }
    if (warp == 1) dev::tmem_alloc<2>(&tmem_at, 512);
    dev::tc_fence_before();
    dev::cluster_sync();  // the pair's barriers and tensor memory are there
    dev::tc_fence_after();
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    const uint32_t tmem = tmem_at;
    auto gave_up = [&] {
        if (!abort_flag) {
            atomicOr(&g_fp4_error_word, 1u);
            abort_flag = 1;
        }
    };

    WideWalk w(p, kWidth);
    if (warp == 0 && lane == 0) {
        auto at = [&](int map) { return (p.moves >> map) & 1u ? w.e : 0; };
        bool dropped = false, ok = true;
        int i = 0;  // stages loaded
        while (ok && w.next()) {
            for (int k = 0; k < p.stages_k; ++k, ++i) {
                const int st = i % S::kStages, round = i / S::kStages;
                if (round > 0 && !dev::mbar_wait_bounded(&empty[st], (round - 1) & 1,
                                                         p.wait_limit_ns, &abort_flag)) {
                    gave_up();
                    ok = false;
                    break;
                }
                const uint32_t bar = dev::peer_addr(dev::smem_addr(&full[st]), 0);
                if (rank == 0) dev::mbar_arrive_expect_tx(&full[st], 4 * S::kCodes);
                dev::mbar_arrive_expect_tx(&landed[st], 3 * S::SF);
                if ((p.inject & FP8BQ_INJECT_DROP_FIRST_LOAD) && i == 0 && blockIdx.x == 0) {
                    dropped = true;
                    continue;
                }
                uint8_t *b = ring + st * S::kStage;
                const int wn = GATED ? w.n0 : w.n0 + (int)rank * 128;
                const int wi = GATED ? (int)rank : 0;
                dev::tma_load_3d_pair(b, &p.x, bar, k * 128, w.m0 + (int)rank * 128, at(0));
                dev::tma_load_3d_pair(b + S::kCodes, &p.w[wi], bar, k * 128, wn, at(2 + 2 * wi));
                b += 2 * S::kCodes;
                dev::tma_load_3d(b, &p.xs, &landed[st], k * (S::SF / 8), w.m0 / 128 + (int)rank,
                                 at(1), false);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    dev::tma_load_3d(b + (1 + h) * S::SF, &p.ws[GATED ? h : 0], &landed[st],
                                     k * (S::SF / 8), w.n0 / 128 + (GATED ? 0 : h),
                                     at(3 + (GATED ? 2 * h : 0)), false);
            }
        }
        // Every copy of both CTAs has landed (a dropped stage's others had the
        // whole wait that ran out for it).
        for (int st = 0; st < S::kStages && st < i; ++st) {
            const int fills = (i - st + S::kStages - 1) / S::kStages;
            if (dropped && st == 0 && fills == 1) continue;
            if ((rank == 0 &&
                 !dev::mbar_wait_bounded(&full[st], (fills - 1) & 1, kDrainNs, nullptr)) ||
                !dev::mbar_wait_bounded(&landed[st], (fills - 1) & 1, kDrainNs, nullptr))
                atomicOr(&g_fp4_error_word, 2u);
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        constexpr uint32_t word = dev::mma_word(FMT, 256, 256);
        bool ok = true;
        int i = 0, n = 0;  // stages, tiles
        for (; ok && w.next(); ++n) {
            if (n > 0 && !dev::mbar_wait_bounded(&drained, (n - 1) & 1, p.wait_limit_ns,
                                                 &abort_flag)) {
                gave_up();
                break;
            }
            dev::tc_fence_after();
            const uint32_t d = tmem + (n & 1) * S::kOther;
            for (int k = 0; k < p.stages_k; ++k, ++i) {
                const int st = i % S::kStages;
                if (!dev::mbar_wait_bounded(&full[st], (i / S::kStages) & 1, p.wait_limit_ns,
                                            &abort_flag) ||
                    !dev::mbar_wait_bounded(&scaled[i % S::kSfBufs], (i / S::kSfBufs) & 1,
                                            p.wait_limit_ns, &abort_flag)) {
                    gave_up();
                    ok = false;
                    break;
                }
                dev::tc_fence_after();
                const uint32_t at = dev::smem_addr(ring + st * S::kStage);
                const uint32_t sx = tmem + S::kScales + (i % S::kSfBufs) * S::kSfCols;
                const uint32_t sw = sx + 4 * S::KT;
                const uint64_t xd = dev::operand_desc(at), wd = dev::operand_desc(at + S::kCodes);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (4 * k + j >= p.mma_k) break;
                    const int t = j * S::KT / 4;
                    dev::mma_fp4<FMT, 2>(
                        d, xd + 2 * j, wd + 2 * j,
                        dev::mma_word_id(word, FMT == FP8BQ_MXFP4 ? 2 * (j & 1) : 0), sx + 4 * t,
                        sw + 8 * t, k + j > 0);
                }
                dev::mma_commit<2>(&empty[st]);
            }
            dev::mma_commit<2>(&sums);
        }
        dev::mma_commit_pair_here(&done);
        if (!dev::mbar_wait_bounded(&done, 0, kDrainNs, nullptr)) atomicOr(&g_fp4_error_word, 2u);
    } else if (warp >= 4 && warp < 8) {
        // Every lane quarter gets the same copy of the scales: lane l of column
        // c holds the four blocks of row l + 32 c, so a lane's 16 bytes of a
        // tile are its words of four columns.
        const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
        bool ok = true;
        for (int i = 0; ok && w.next();) {
            for (int k = 0; k < p.stages_k; ++k, ++i) {
                const int st = i % S::kStages, b = i % S::kSfBufs;
                bool here = dev::mbar_wait_bounded(&landed[st], (i / S::kStages) & 1,
                                                   p.wait_limit_ns, &abort_flag);
                const uint8_t *sf = ring + st * S::kStage + 2 * S::kCodes + lane * 16;
                uint4 v[3 * S::KT];  // of the tokens, then tile by tile of the weight's two rows
#pragma unroll
                for (int t = 0; t < S::KT; ++t) {
                    v[t] = *(const uint4 *)(sf + t * kFp4TileBytes);
                    v[S::KT + 2 * t] = *(const uint4 *)(sf + S::SF + t * kFp4TileBytes);
                    v[S::KT + 2 * t + 1] = *(const uint4 *)(sf + 2 * S::SF + t * kFp4TileBytes);
                }
                if (i >= S::kSfBufs) {  // the products that read this buffer are done
                    const int o = i - S::kSfBufs;
                    here = here && dev::mbar_wait_bounded(&empty[o % S::kStages],
                                                          (o / S::kStages) & 1, p.wait_limit_ns,
                                                          &abort_flag);
                }
                if (!__all_sync(0xffffffffu, here)) {
                    if (lane == 0) gave_up();
                    ok = false;
                    break;
                }
                dev::tc_fence_after();
#pragma unroll
                for (int t = 0; t < 3 * S::KT; t += 2)
                    dev::tmem_st8(tmem + quarter + S::kScales + b * S::kSfCols + 4 * t, v[t], v[t + 1]);
                dev::tmem_st_wait();
                dev::tc_fence_before();
                __syncwarp();
                if (lane == 0) dev::peer_arrive(dev::peer_addr(dev::smem_addr(&scaled[b]), 0));
            }
        }
    } else if (warp >= 8) {
        const int quarter = warp & 3, half = (warp - 8) >> 2;
        const uint32_t drained_bar = dev::peer_addr(dev::smem_addr(&drained), 0);
        for (int n = 0; w.next(); ++n) {
            const bool here =
                dev::mbar_wait_bounded(&sums, n & 1, 2 * p.wait_limit_ns, &abort_flag);
            if (!__all_sync(0xffffffffu, here)) {
                if (lane == 0) gave_up();
                break;
            }
            dev::tc_fence_after();
            const uint32_t d = tmem + (n & 1) * S::kOther + ((uint32_t)(quarter * 32) << 16);
            const int64_t m = w.m0 + (int)rank * 128 + quarter * 32 + lane;
            const bool in = m < w.valid;
            const float xt = MM_XT(p, w.e), alpha = __fmul_rn(xt, MM_WT(p, 0, w.e));
            const float alpha1 = GATED ? __fmul_rn(xt, MM_WT(p, 1, w.e)) : 0.0f;
            // runs of 32 columns, the shared ones (5-7 of even tiles, 0-2 of
            // odd ones) first; the two warps of a quarter take turns
            constexpr int kRuns = GATED ? 4 : 8;
#pragma unroll 1
            for (int j = half; j < kRuns; j += 2) {
                const int c = (n & 1) ? j : kRuns - 1 - j;
                float v[32];
                if constexpr (GATED) {
                    uint32_t g[32], u[32];
                    dev::tmem_ld32(d + 32 * c, g);
                    dev::tmem_ld32(d + 128 + 32 * c, u);
                    dev::tmem_ld_wait();
                    if (j == 2 - half) {  // its last run of the first three
                        dev::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) dev::peer_arrive(drained_bar);
                    }
#pragma unroll
                    for (int q = 0; q < 32; ++q)
                        v[q] = silu(__uint_as_float(g[q]) * alpha) * (__uint_as_float(u[q]) * alpha1);
                } else {
                    uint32_t g[32];
                    dev::tmem_ld32(d + 32 * c, g);
                    dev::tmem_ld_wait();
                    if (j == 2 - half) {  // its last run of the first three
                        dev::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) dev::peer_arrive(drained_bar);
                    }
#pragma unroll
                    for (int q = 0; q < 32; ++q) v[q] = __uint_as_float(g[q]) * alpha;
                }
                if (in && w.n0 + 32 * c < p.N) store32<BF16>(p, w.e, m, w.n0 + 32 * c, v);
            }
        }
    }
    __syncwarp();
    dev::tc_fence_before();
    dev::cluster_sync();  // no access to this CTA's memory is left
    if (warp == 1) dev::tmem_dealloc<2>(tmem, 512);
}

template <typename K>
cudaError_t set_smem(K kernel, int smem) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

template <typename K>
cudaError_t launch_clusters(K kern, dim3 grid, unsigned threads, unsigned cluster, int smem,
                            cudaStream_t st, const Fp4MmParams &p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int FMT, bool GATED, bool BF16, int NT>
cudaError_t narrow(const Fp4MmParams &p0, cudaStream_t st) {
    using S = Narrow<FMT, GATED, NT>;
    auto kern = k_fp4_narrow<FMT, GATED, BF16, NT>;
    static PerDevice<cudaError_t> setup;
    const cudaError_t e = setup.get([&] { return set_smem(kern, S::kSmem); });
    if (e != cudaSuccess) return e;
    Fp4MmParams p = p0;
    const int64_t nt = (p.N + 127) / 128, mt = (p.M + NT - 1) / NT;
    const int64_t tiles = nt * mt * p.batch;
    // CTAs that fit at once, shared out over the tiles: the cluster's size
    const int64_t slots = (int64_t)sm_count() * (S::kSmem == S::kSmall ? 2 : 1);
    int64_t split = slots / tiles;
    split = split < 1 ? 1 : split > 8 ? 8 : split;
    p.split = (int32_t)(split > p.stages_k ? p.stages_k : split);
    return launch_clusters(kern, dim3((unsigned)(nt * p.split), (unsigned)mt, (unsigned)p.batch),
                           128, (unsigned)p.split, S::kSmem, st, p);
}

template <int FMT, bool GATED, bool BF16>
cudaError_t narrow_tokens(const Fp4MmParams &p, int tokens, cudaStream_t st) {
    switch (tokens) {
        case 16: return narrow<FMT, GATED, BF16, 16>(p, st);
        case 32: return narrow<FMT, GATED, BF16, 32>(p, st);
        case 64: return narrow<FMT, GATED, BF16, 64>(p, st);
        case 128: return narrow<FMT, GATED, BF16, 128>(p, st);
        default:
            if constexpr (GATED) return cudaErrorInvalidValue;
            else return narrow<FMT, GATED, BF16, 256>(p, st);
    }
}

template <int FMT>
cudaError_t narrow_format(const Fp4MmParams &p, bool gated, bool bf16, int tokens,
                          cudaStream_t st) {
    if (gated)
        return bf16 ? narrow_tokens<FMT, true, true>(p, tokens, st)
                    : narrow_tokens<FMT, true, false>(p, tokens, st);
    return bf16 ? narrow_tokens<FMT, false, true>(p, tokens, st)
                : narrow_tokens<FMT, false, false>(p, tokens, st);
}

template <int FMT, bool GATED, bool BF16>
cudaError_t wide(const Fp4MmParams &p, cudaStream_t st) {
    using S = Wide<FMT>;
    auto kern = k_fp4_wide<FMT, GATED, BF16>;
    static PerDevice<cudaError_t> setup;
    const cudaError_t e = setup.get([&] { return set_smem(kern, S::kSmem); });
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)((p.M + 255) / 256) * ((p.N + (GATED ? 127 : 255)) / (GATED ? 128 : 256)) *
                          p.batch;
    const int64_t pairs = sm_count() / 2;
    return launch_clusters(kern, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), S::kThreads, 2,
                           S::kSmem, st, p);
}

template <int FMT>
cudaError_t wide_format(const Fp4MmParams &p, bool gated, bool bf16, cudaStream_t st) {
    if (gated) return bf16 ? wide<FMT, true, true>(p, st) : wide<FMT, true, false>(p, st);
    return bf16 ? wide<FMT, false, true>(p, st) : wide<FMT, false, false>(p, st);
}

}  // namespace

cudaError_t launch_fp4_mm_wide(const Fp4MmParams &p, int format, bool gated, bool out_bf16,
                               cudaStream_t st) {
    return format == FP8BQ_MXFP4 ? wide_format<FP8BQ_MXFP4>(p, gated, out_bf16, st)
                                 : wide_format<FP8BQ_NVFP4>(p, gated, out_bf16, st);
}

int fp4_narrow_tokens(int64_t M, bool gated) {
    for (int t : {16, 32, 64, 128})
        if (M <= t) return t;
    return gated ? 128 : 256;
}

cudaError_t launch_fp4_mm_narrow(const Fp4MmParams &p, int format, bool gated, bool out_bf16,
                                 int tokens, cudaStream_t st) {
    return format == FP8BQ_MXFP4 ? narrow_format<FP8BQ_MXFP4>(p, gated, out_bf16, tokens, st)
                                 : narrow_format<FP8BQ_NVFP4>(p, gated, out_bf16, tokens, st);
}

cudaError_t read_and_clear_fp4_error_word(uint32_t *out) {
    uint32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_fp4_error_word, sizeof(uint32_t));
    if (e != cudaSuccess) return e;
    if (*out) e = cudaMemcpyToSymbol(g_fp4_error_word, &zero, sizeof(uint32_t));
    return e;
}

FP8BQ_DEFINE_BOUNDS_RECORD(bounds_record_fp4_mm)

}  // namespace fp8bq
