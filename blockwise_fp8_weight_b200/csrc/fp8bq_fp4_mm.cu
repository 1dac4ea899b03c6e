// fp8bq_fp4_mm.cu -- products of 4-bit matrices on the block-scaled tensor
// cores: out = a b^T, and out = silu(a b^T) * (a up^T).
//
// The codes go from memory to shared memory as they are (TMA, 128-byte
// swizzle: 256 codes of a row), the scale tiles too; a scale tile is copied
// into tensor memory next to the fp32 sums, and tcgen05.mma multiplies codes
// and scales of 64 columns of K at a time.  Nothing is unpacked.
#include <atomic>

#include "fp8bq_fp4_device.cuh"

namespace fp8bq {

// Bits as in the TMA quantiser's error word: 1 a wait ran out, 2 a copy or a
// product may still be in flight.
__device__ uint32_t g_fp4_error_word;
// Whether a product was launched or captured: until then the word is not read
// (10 us a read, and the first one would load these kernels, 11 ms).
static std::atomic<bool> g_fp4_launched{false};

namespace {

constexpr uint64_t kDrainNs = 2000000000ull;

#define MM_SPAN(base, bytes) (dev::Span{(uint64_t)(base), (uint64_t)(base) + (bytes)})

// silu(v) = v / (1 + exp(-v)) with e = exp(-|v|) <= 1: v / (1 + e) from zero on,
// v e / (1 + e) below, so that nothing overflows on the way and the fast
// division, whose divisor is in [1, 2], is off by 2 units of 2^-23 at most.
// The exponential: expf for fp32 outputs (2 units); for bf16 outputs the fast
// one, whose documented error of 2 + 1.173 |v| units is far below their
// rounding.  Measured on B200, gated mxfp4, 8192 x 6144 outputs: K = 512 fp32 80
// us (the fast one: 63), bf16 63; K = 4096 no difference.
template <bool BF16>
__device__ __forceinline__ float silu(float v) {
    const float e = BF16 ? __expf(-fabsf(v)) : expf(-fabsf(v));
    return __fdividef(v < 0.0f ? v * e : v, 1.0f + e);
}

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

// A place in a ring of N slots and the parity of its round.
template <int N>
struct Slot {
    int at = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++at == N) {
            at = 0;
            parity ^= 1;
        }
    }
};

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

// Scales of a stage into tensor memory, by one warp for its lane quarter.  A
// scale tile takes four columns; lane l of column c holds the four blocks of
// row l + 32 c, so a lane's 16 bytes of a tile are its words of the columns,
// and every quarter gets the same copy.  The scales go through registers
// (ld.shared, tcgen05.st) rather than by tcgen05.cp: a copy of one tile holds
// up the tensor cores for 62 clocks.
template <int TILES>
__device__ __forceinline__ void scales_to_tmem(uint32_t dst, const uint4 (&v)[TILES]) {
    static_assert(TILES % 2 == 0, "pairs of tiles");
#pragma unroll
    for (int t = 0; t < TILES; t += 2) dev::tmem_st8(dst + 4 * t, v[t], v[t + 1]);
    dev::tmem_st_wait();
}

// ============================================================== few tokens
//
// A CTA computes 128 outputs (rows of the weight, the M side of the tensor
// core's tile) for NT tokens (its N side; tiles of 16 and 32 only where they
// hold all tokens: scale tiles begin every 128): few tokens cost few MMA columns,
// and the kernel is bound by the weight's bytes.
//
// Where the tiles are too few to keep every SM loading, a cluster of `split`
// CTAs shares a tile: each sums a run of K, the partial sums meet in shared
// memory, and every CTA of the cluster adds up and stores a part of the tile,
// in the order of the ranks: no atomics, no workspace, the same sum every
// time.  Otherwise (split == 1) a CTA walks over tiles, and loads and
// multiplies the next one while it stores.
//
// Warp 0 loads (one lane), warp 1 issues the products (one lane), warps 4-7
// bring the scales into tensor memory, warps 8-11 store.  Every wait is
// bounded; one that runs out sets the error word, and the CTA still waits for
// its copies and products before it leaves.
template <int FMT, bool GATED, int NT>
struct Narrow {
    static constexpr int W = GATED ? 2 : 1;
    static constexpr int KT = 256 / (4 * fp4_block(FMT));   // scale tiles along a stage's K
    static constexpr int SF = KT * kFp4TileBytes;           // scales of 128 rows
    static constexpr int XT = (NT + 127) / 128;             // token scale tile rows
    static constexpr int kCodesW = 128 * 128;
    static constexpr int kCodesX = NT * 128;
    static constexpr int kStage = W * (kCodesW + SF) + kCodesX + XT * SF;
    static constexpr int kTiles = KT * (W + XT);            // scale tiles of a stage
    static constexpr int kSfCols = 4 * kTiles;
    // Sums of two tiles where they fit beside two stages' scales.
    static constexpr int kSums = W * NT;
    static constexpr int kAcc = 2 * kSums + 2 * kSfCols <= 512 ? 2 : 1;
    // Two CTAs an SM where their sums and rings leave room, else one.  A CTA
    // that takes c of the 512 tensor-memory columns takes at least c / 512 of
    // the SM's shared memory, so CTAs that share an SM always find their
    // columns and none waits for another's while a third waits for it.
    static constexpr int kSmall = 114688, kLarge = 231424;  // 112 KB, 226 KB
    static constexpr bool kTwo =
        kAcc * kSums + 2 * kSfCols <= 256 && 2 * kStage + 1024 <= kSmall;
    static constexpr int kCols = kTwo ? 256 : 512;
    static constexpr int kSmem = kTwo ? kSmall : kLarge;
    static constexpr int kStages = (kSmem - 1024) / kStage;
    static constexpr int kFit = (kCols - kAcc * kSums) / kSfCols;
    static constexpr int kSfBufs = kFit < kStages ? kFit : kStages;
    static constexpr int kThreads = 384;
    static_assert(kStages >= 2 && kSfBufs >= 2, "ring");
    static_assert(kSums * 128 * 4 <= kStages * kStage, "partial sums");
};

// The tiles of a CTA (of its cluster), the same for every role; tiles without
// valid rows are passed over.  The weight's rows run fastest.
struct NarrowWalk {
    const Fp4MmParams &p;
    uint32_t t, step, total, mt, nt;  // fewer than 2^31 tiles (checked on the host)
    int width, m0, n0, e, valid;
    bool placed;  // (m0, n0, e) is tile t's
    // The first tile's place is found here, ahead of the wait for the previous
    // kernel: `rows` may be what that kernel writes, and is read by next().
    __device__ __forceinline__ NarrowWalk(const Fp4MmParams &q, int width_)
        : p(q), step(gridDim.x), width(width_), placed(true) {
        t = blockIdx.x;
        if (p.split > 1) {  // a cluster for each tile
            t /= (uint32_t)p.split;
            step /= (uint32_t)p.split;
        }
        mt = (uint32_t)(p.M + width - 1) / (uint32_t)width;
        nt = (uint32_t)(p.N + 127) / 128;
        total = mt * nt * (uint32_t)p.batch;
        place();
    }
    __device__ __forceinline__ void place() {
        uint32_t r = 0;
        n0 = (int)t;
        if (t >= nt) {
            r = t / nt;
            n0 = (int)(t - r * nt);
        }
        n0 *= 128;
        e = mt == 1 ? (int)r : (int)(r / mt);
        m0 = (int)(r - (uint32_t)e * mt) * width;
    }
    __device__ __forceinline__ bool next() {
        for (; t < total; t += step) {
            if (!placed) place();
            placed = false;
            valid = min(width, valid_rows(p, e) - m0);
            if (valid > 0) {
                t += step;
                return true;
            }
        }
        return false;
    }
};

// A cluster's partial sums of one tile added up and stored: every CTA takes
// vectors of four outputs in turn, and adds them in the order of the ranks.
// B >= split: eight loads from the peers are under way at a time, of one or
// several vectors.
template <int B, int W, int NT, int THREADS, bool BF16>
__device__ __forceinline__ void add_parts(const Fp4MmParams &p, const NarrowWalk &w, uint32_t base,
                                          int rank) {
    constexpr int V = 8 / B;
    const float xt = MM_XT(p, w.e);
    float alpha[W];
#pragma unroll
    for (int u = 0; u < W; ++u) alpha[u] = __fmul_rn(xt, MM_WT(p, u, w.e));
    const int vecs = w.valid * 32, step = p.split * THREADS;
    for (int q0 = rank * THREADS + (int)threadIdx.x; q0 < vecs; q0 += V * step) {
        float v[V][W][4];
#pragma unroll
        for (int u = 0; u < W; ++u) {
            float4 f[V][B];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int q = q0 + i * step;
                const uint32_t a = base + ((u * NT + (q >> 5)) * 128 + (q & 31) * 4) * 4;
#pragma unroll
                for (int r = 0; r < B; ++r)
                    if (r < p.split && q < vecs) f[i][r] = dev::peer_ld4(dev::peer_addr(a, r));
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float4 s = f[i][0];
#pragma unroll
                for (int r = 1; r < B; ++r)
                    if (r < p.split) {
                        s.x += f[i][r].x, s.y += f[i][r].y;
                        s.z += f[i][r].z, s.w += f[i][r].w;
                    }
                v[i][u][0] = s.x * alpha[u], v[i][u][1] = s.y * alpha[u];
                v[i][u][2] = s.z * alpha[u], v[i][u][3] = s.w * alpha[u];
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int q = q0 + i * step, o = w.n0 + (q & 31) * 4;
            if (q >= vecs || o >= p.N) continue;
            if constexpr (W == 2)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][0][j] = silu<BF16>(v[i][0][j]) * v[i][W - 1][j];
            store4<BF16>(p, w.e, w.m0 + (q >> 5), o, v[i][0]);
        }
    }
}

template <int FMT, bool GATED, bool BF16, int NT>
__global__ void __launch_bounds__(384, Narrow<FMT, GATED, NT>::kTwo ? 2 : 1)
    k_fp4_narrow(const __grid_constant__ Fp4MmParams p) {
    using S = Narrow<FMT, GATED, NT>;
    constexpr int ES = BF16 ? 2 : 4;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages], scaled[S::kSfBufs];
    __shared__ __align__(8) uint64_t sums[S::kAcc], freed[S::kAcc], done;
    __shared__ uint32_t tmem_at;
    __shared__ volatile int abort_flag;
    uint8_t *ring = raw + ((1024u - (dev::smem_addr(raw) & 1023u)) & 1023u);

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same for a warp
    const uint32_t split = (uint32_t)p.split, rank = split > 1 ? dev::cluster_rank() : 0;
    int k0 = 0, k1 = p.stages_k;  // this CTA's stages (fewer than 2^23)
    if (split > 1) {
        k0 = (int)((uint32_t)p.stages_k * rank / split);
        k1 = (int)((uint32_t)p.stages_k * (rank + 1) / split);
    }
    if (tid == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            dev::mbar_init(&full[s], 1);
            dev::mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < S::kSfBufs; ++s) dev::mbar_init(&scaled[s], 4);
        for (int s = 0; s < S::kAcc; ++s) {
            dev::mbar_init(&sums[s], 1);
            dev::mbar_init(&freed[s], 4);
        }
        dev::mbar_init(&done, 1);
        abort_flag = 0;
        dev::fence_mbar_init();
        dev::prefetch_tensormap(&p.x);  // that of the scales as well costs 0.3 us
    }
    if (warp == 1) dev::tmem_alloc<1>(&tmem_at, S::kCols);
    NarrowWalk w(p, NT);
    auto at = [&](int map) { return (p.moves >> map) & 1u ? w.e : 0; };
    if (warp == 2 && lane == 0) {  // the weight's first stages on their way to L2
        for (int k = k0; k < k1 && k < k0 + S::kStages; ++k)
#pragma unroll
            for (int v = 0; v < S::W; ++v) {
                dev::tma_prefetch_3d(&p.w[v], k * 128, w.n0, at(2 + 2 * v));
                dev::tma_prefetch_3d(&p.ws[v], k * (S::SF / 8), w.n0 / 128, at(3 + 2 * v));
            }
    }
    dev::tc_fence_before();
    __syncthreads();
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
    float *part = reinterpret_cast<float *>(ring);  // [weight][token][128 outputs]
    // Every other 16 columns of this warp's lanes of the sums to `part`.  (The
    // ring is free: every stage was multiplied.)
    auto to_part = [&](int valid, int first) {
        const uint32_t d = tmem + ((uint32_t)((warp & 3) * 32) << 16);
#pragma unroll
        for (int c = 0; c < S::kSums; c += 16) {
            if (c % NT >= valid || (c / 16 & 1) != first) continue;
            uint32_t v[16];
            dev::tmem_ld16(d + c, v);
            dev::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j)
                part[(c + j) * 128 + (warp & 3) * 32 + lane] = __uint_as_float(v[j]);
        }
    };

    if (warp == 0 && dev::elect_one()) {
        bool dropped = false, ok = true;
        int i = 0;  // stages loaded
        Slot<S::kStages> s;
        while (ok && w.next()) {
            for (int k = k0; k < k1; ++k, ++i, s.next()) {
                const int st = s.at;
                if (i >= S::kStages && !dev::mbar_wait_bounded(&empty[st], s.parity ^ 1,
                                                               p.wait_limit_ns, &abort_flag)) {
                    gave_up();
                    ok = false;
                    break;
                }
                dev::mbar_arrive_expect_tx(&full[st], S::kStage);
                if ((p.inject & FP8BQ_INJECT_DROP_FIRST_LOAD) && i == 0 && blockIdx.x == 0) {
                    dropped = true;
                    continue;
                }
                uint8_t *b = ring + st * S::kStage;
#pragma unroll
                for (int v = 0; v < S::W; ++v, b += S::kCodesW)
                    dev::tma_load_3d(b, &p.w[v], &full[st], k * 128, w.n0, at(2 + 2 * v), false);
                dev::tma_load_3d(b, &p.x, &full[st], k * 128, w.m0, at(0), false);
                b += S::kCodesX;
#pragma unroll
                for (int v = 0; v < S::W; ++v, b += S::SF)
                    dev::tma_load_3d(b, &p.ws[v], &full[st], k * (S::SF / 8), w.n0 / 128,
                                     at(3 + 2 * v), false);
#pragma unroll
                for (int t = 0; t < S::XT; ++t, b += S::SF)
                    dev::tma_load_3d(b, &p.xs, &full[st], k * (S::SF / 8), w.m0 / 128 + t, at(1),
                                     false);
            }
        }
        for (int st = 0; st < S::kStages && st < i; ++st) {  // every copy has landed
            const int fills = (i - st + S::kStages - 1) / S::kStages;
            if (dropped && st == 0 && fills == 1) continue;
            if (!dev::mbar_wait_bounded(&full[st], (fills - 1) & 1, kDrainNs, nullptr))
                atomicOr(&g_fp4_error_word, 2u);
        }
    } else if (warp == 1 && dev::elect_one()) {
        constexpr uint32_t word = dev::mma_word(FMT, 128, NT);
        bool ok = true;
        int n = 0;  // tiles
        Slot<S::kStages> s;
        Slot<S::kSfBufs> f;
        bool ready = false;
        Slot<S::kAcc> acc;
        const uint64_t first = dev::operand_desc(dev::smem_addr(ring));
        for (; ok && w.next(); ++n, acc.next()) {
            if (n >= S::kAcc && !dev::mbar_wait_bounded(&freed[acc.at], acc.parity ^ 1,
                                                        p.wait_limit_ns, &abort_flag)) {
                gave_up();
                break;
            }
            const uint32_t d = tmem + acc.at * S::kSums;
            for (int k = k0; k < k1; ++k, s.next()) {
                const uint64_t wd = first + (uint32_t)(s.at * (S::kStage >> 4));
                const uint64_t xd = wd + (S::W * S::kCodesW >> 4);
                const uint32_t sw = tmem + S::kAcc * S::kSums + f.at * S::kSfCols;
                // tokens 64-127 of a scale tile begin at its third column
                const uint32_t sx = sw + 4 * S::KT * S::W + (NT == 64 ? (w.m0 & 64) >> 5 : 0);
                const int steps = p.mma_k - 4 * k;  // 64-column steps left
                if (!ready && !dev::mbar_wait_bounded(&scaled[f.at], f.parity, p.wait_limit_ns,
                                                      &abort_flag)) {
                    gave_up();
                    ok = false;
                    break;
                }
                dev::tc_fence_after();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j >= steps) break;
                    const int t = j * S::KT / 4;
#pragma unroll
                    for (int v = 0; v < S::W; ++v)
                        dev::mma_fp4<FMT, 1>(
                            d + v * NT, wd + (v * S::kCodesW >> 4) + 2 * j, xd + 2 * j,
                            dev::mma_word_id(word, FMT == FP8BQ_MXFP4 ? 2 * (j & 1) : 0),
                            sw + 4 * (v * S::KT + t), sx + 4 * t * S::XT, j > 0 || k > k0);
                }
                f.next();
                ready = dev::mbar_try_wait(&scaled[f.at], f.parity);  // the next stage's
                dev::mma_commit<1>(&empty[s.at]);
            }
            dev::mma_commit<1>(&sums[acc.at]);
        }
        dev::mma_commit<1>(&done);
        if (!dev::mbar_wait_bounded(&done, 0, kDrainNs, nullptr)) atomicOr(&g_fp4_error_word, 2u);
    } else if (warp >= 4 && warp < 8) {
        const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
        bool ok = true;
        Slot<S::kStages> s, old;  // `old`: kSfBufs stages behind
        Slot<S::kSfBufs> f;
        for (int i = 0; ok && w.next();) {
            for (int k = k0; k < k1; ++k, ++i, s.next(), f.next()) {
                bool here = dev::mbar_wait_bounded(&full[s.at], s.parity, p.wait_limit_ns,
                                                   &abort_flag);
                const uint8_t *sf =
                    ring + s.at * S::kStage + S::W * S::kCodesW + S::kCodesX + lane * 16;
                uint4 v[S::kTiles];  // of each weight, then tile by tile of the tokens
#pragma unroll
                for (int t = 0; t < S::KT; ++t) {
#pragma unroll
                    for (int u = 0; u < S::W; ++u)
                        v[u * S::KT + t] = *(const uint4 *)(sf + u * S::SF + t * kFp4TileBytes);
#pragma unroll
                    for (int x = 0; x < S::XT; ++x)
                        v[S::W * S::KT + t * S::XT + x] =
                            *(const uint4 *)(sf + (S::W + x) * S::SF + t * kFp4TileBytes);
                }
                if (i >= S::kSfBufs) {  // the products that read this buffer are done
                    here = here && dev::mbar_wait_bounded(&empty[old.at], old.parity,
                                                          p.wait_limit_ns, &abort_flag);
                    old.next();
                }
                if (!__all_sync(0xffffffffu, here)) {
                    if (lane == 0) gave_up();
                    ok = false;
                    break;
                }
                dev::tc_fence_after();
                scales_to_tmem<S::kTiles>(
                    tmem + quarter + S::kAcc * S::kSums + f.at * S::kSfCols, v);
                dev::tc_fence_before();
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(&scaled[f.at]);
            }
        }
        if (split > 1 && ok && S::kSums > 16 && w.valid > 0) {  // the tile's other half
            const bool here =
                dev::mbar_wait_bounded(&sums[0], 0, 2 * p.wait_limit_ns, &abort_flag);
            if (__all_sync(0xffffffffu, here)) {
                dev::tc_fence_after();
                to_part(w.valid, 1);
            } else if (lane == 0) {
                gave_up();
            }
        }
    } else if (warp >= 8) {
        const int row = (warp & 3) * 32 + lane;  // of the weight's 128
        for (Slot<S::kAcc> acc; w.next(); acc.next()) {
            const bool here = dev::mbar_wait_bounded(&sums[acc.at], acc.parity,
                                                     2 * p.wait_limit_ns, &abort_flag);
            if (!__all_sync(0xffffffffu, here)) {
                if (lane == 0) gave_up();
                break;
            }
            dev::tc_fence_after();
            const uint32_t d = tmem + acc.at * S::kSums + ((uint32_t)((warp & 3) * 32) << 16);
            if (split > 1) {
                to_part(w.valid, 0);
                continue;
            }
            const float xt = MM_XT(p, w.e), alpha = __fmul_rn(xt, MM_WT(p, 0, w.e));
            const float alpha1 = GATED ? __fmul_rn(xt, MM_WT(p, 1, w.e)) : 0.0f;
            const int o = w.n0 + row;
            char *dst = (char *)p.out + (w.e * p.obs + (int64_t)w.m0 * p.ldo + o) * ES;
#pragma unroll 1
            for (int c = 0; c < w.valid; c += 16) {
                uint32_t g[16], u[16];
                dev::tmem_ld16(d + c, g);
                if constexpr (GATED) dev::tmem_ld16(d + NT + c, u);
                dev::tmem_ld_wait();
                if (c + 16 >= w.valid) {
                    dev::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) dev::mbar_arrive(&freed[acc.at]);
                }
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    v[j] = __uint_as_float(g[j]) * alpha;
                    if constexpr (GATED) v[j] = silu<BF16>(v[j]) * (__uint_as_float(u[j]) * alpha1);
                }
                if (NT == 16 && BF16 && p.store_align >= 4) {
                    // two tokens at a time: an even lane stores its and its
                    // neighbour's output of the first, an odd one of the second
                    // (16 tokens against 151936 x 512 on B200: 7.2 us, by element
                    // 7.8; wider tiles are 5 to 30 % slower this way)
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const bool odd = lane & 1;
                        const float get =
                            __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
                        const uint32_t two = odd ? bf16x2(get, v[j + 1]) : bf16x2(v[j], get);
                        const int t = c + j + odd;
                        char *q = dst + (t * p.ldo - odd) * ES;
                        if (t < w.valid && (o | 1) < p.N) {
                            if (FP8BQ_IN(MM_SPAN(p.out, p.out_bytes), q, 4)) *(uint32_t *)q = two;
                        } else if (t < w.valid && (o & ~1) < p.N &&
                                   FP8BQ_IN(MM_SPAN(p.out, p.out_bytes), q, 2)) {
                            *(uint16_t *)q = (uint16_t)two;
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        char *q = dst + (c + j) * p.ldo * ES;
                        if (c + j < w.valid && o < p.N &&
                            FP8BQ_IN(MM_SPAN(p.out, p.out_bytes), q, ES)) {
                            if constexpr (BF16) *(uint16_t *)q = (uint16_t)bf16x2(v[j], 0.0f);
                            else *(float *)q = v[j];
                        }
                    }
                }
            }
        }
    }
    __syncwarp();
    dev::tc_fence_before();
    if (split > 1) {
        NarrowWalk one(p, NT);
        if (one.next()) {  // the same for every CTA of a cluster
            dev::cluster_sync();
            const uint32_t base = dev::smem_addr(part);
            // few tokens: one way only, a short kernel starts sooner
            if (!abort_flag) {
                if (NT >= 64 && split <= 2)
                    add_parts<2, S::W, NT, S::kThreads, BF16>(p, one, base, rank);
                else
                    add_parts<8, S::W, NT, S::kThreads, BF16>(p, one, base, rank);
            }
            dev::cluster_sync();  // peers may still read this CTA's sums
        }
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
// warps 4-7 and 16-19 bring the scales of every other stage into tensor memory
// (one group of four needs about 700 clocks a stage beside 512 of products, by
// the latency of its waits and instructions: 91 us instead of 83, nvfp4 102
// instead of 90), warps 8-15 store; warp 1 of
// the first CTA issues the products of both.  The sums of successive tiles
// alternate between columns [0, 256) and [160, 416), so the next tile is
// multiplied while this one is stored; the 96 columns that both use are read
// first, and the next tile waits for those alone.  The scales' buffers take
// the last 96 columns.
//
// Measured on B200, 8192 tokens against 6144 x 4096 (mxfp4 / nvfp4): 82 / 88 us;
// with the scales copied by tcgen05.cp, 6 or 12 tiles a stage beside 768
// clocks of products, before the other steps: 133 / 171 against 107 / 110.
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
    static constexpr int kThreads = 640;
    static constexpr int kStore = 1024;                        // a storing warp's, of eight
    static_assert(kSfBufs >= 2 && kSfBufs <= kStages, "scale buffers");
    static_assert(1024 + kStages * kStage + 8 * kStore <= kSmem, "room to store");
};

// 16 consecutive outputs of a row, from column n; rows begin at multiples of 16
// bytes (fp32: 32).
template <bool BF16>
__device__ __forceinline__ void store16(const Fp4MmParams &p, int64_t e, int64_t m, int n,
                                        const float (&v)[16]) {
    constexpr int ES = BF16 ? 2 : 4, PER = 32 / ES;            // outputs in 32 bytes
    char *dst = (char *)p.out + (e * p.obs + m * p.ldo + n) * ES;
#pragma unroll
    for (int c = 0; c < 16; c += PER, dst += 32) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = BF16 ? bf16x2(v[(c + 2 * j) & 15], v[(c + 2 * j + 1) & 15])
                        : __float_as_uint(v[(c + j) & 15]);
        if (n + c + PER <= p.N) {
            if (!FP8BQ_IN(MM_SPAN(p.out, p.out_bytes), dst, 32)) continue;
            if (!BF16 || p.store_align >= 32) {
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

// The same of a warp's 32 rows from row m, `rows` of them to be stored, where
// rows begin at multiples of W bytes only: 32 bytes a row at a time through
// shared memory, so that a store covers 32 bytes of W rows rather than W of 32.
// Measured on B200, 8192 tokens, K = 512, and with every lane storing its own
// row: 6148 fp32 outputs (W = 16) 81 us, 127; 6143 (W = 4) 112, 350; 6148 bf16
// outputs (4) 47, 470; 6143 (2) 62, 470.  (6152 bf16 outputs, 16: 37, 40, but
// gated 70, 62; 6144 fp32 outputs, 32: 64, 51.  Those the lanes store.)
template <bool BF16, int W>
__device__ __forceinline__ void store_pieces(const Fp4MmParams &p, int64_t e, int64_t m, int rows,
                                             int n, const char *buf, int lane) {
    constexpr int ES = BF16 ? 2 : 4;
    const int r = lane / (32 / W), c = lane % (32 / W) * W / ES;
    char *dst = (char *)p.out + (e * p.obs + (m + r) * p.ldo + n + c) * ES;
    buf += lane * W;
#pragma unroll
    for (int j = 0; j < 32; j += W, buf += 32 * W, dst += (int64_t)W * p.ldo * ES) {
        if (j + r >= rows) break;
        if (n + c + W / ES <= p.N) {
            if (!FP8BQ_IN(MM_SPAN(p.out, p.out_bytes), dst, W)) continue;
            if constexpr (W == 16) *(uint4 *)dst = *(const uint4 *)buf;
            else if constexpr (W == 4) *(uint32_t *)dst = *(const uint32_t *)buf;
            else *(uint16_t *)dst = *(const uint16_t *)buf;
        } else {
#pragma unroll
            for (int q = 0; q < W / ES; ++q)
                if (n + c + q < p.N && FP8BQ_IN(MM_SPAN(p.out, p.out_bytes), dst + q * ES, ES)) {
                    if constexpr (BF16)
                        *(uint16_t *)(dst + 2 * q) = *(const uint16_t *)(buf + 2 * q);
                    else
                        *(uint32_t *)(dst + 4 * q) = *(const uint32_t *)(buf + 4 * q);
                }
        }
    }
}
template <bool BF16, int W>
__device__ __forceinline__ void store16_staged(const Fp4MmParams &p, int64_t e, int64_t m, int rows,
                                               int n, const float (&v)[16], char *buf, int lane) {
    constexpr int PER = BF16 ? 16 : 8;                         // outputs in 32 bytes
#pragma unroll
    for (int c = 0; c < 16; c += PER) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = BF16 ? bf16x2(v[(c + 2 * j) & 15], v[(c + 2 * j + 1) & 15])
                        : __float_as_uint(v[(c + j) & 15]);
        __syncwarp();  // the last piece is read
        *(uint4 *)(buf + lane * 32) = make_uint4(w[0], w[1], w[2], w[3]);
        *(uint4 *)(buf + lane * 32 + 16) = make_uint4(w[4], w[5], w[6], w[7]);
        __syncwarp();
        store_pieces<BF16, W>(p, e, m, rows, n + c, buf, lane);
    }
}

// The tiles of a pair: first rows, first outputs and matrix of the stack, in
// the same order for every role; tiles without valid rows are passed over.
struct WideWalk {
    const Fp4MmParams &p;
    uint32_t t, step, total, mt, nt;  // fewer than 2^31 tiles (checked on the host)
    int width, m0, n0, e, valid;
    __device__ __forceinline__ WideWalk(const Fp4MmParams &q, int width_)
        : p(q), t(blockIdx.x >> 1), step(gridDim.x >> 1), width(width_) {
        mt = (uint32_t)(p.M + 255) / 256;
        nt = (uint32_t)(p.N + width - 1) / (uint32_t)width;
        total = mt * nt * (uint32_t)p.batch;
    }
    __device__ __forceinline__ bool next() {
        for (; t < total; t += step) {
            const uint32_t r = t / mt;
            e = (int)(r / nt);
            m0 = (int)(t - r * mt) * 256;
            n0 = (int)(r - (uint32_t)e * nt) * width;
            valid = valid_rows(p, e);
            if (m0 < valid) {
                t += step;
                return true;
            }
        }
        return false;
    }
};

// ALIGN: rows of the output begin at multiples of so many bytes, or of more.
template <int FMT, bool GATED, bool BF16, int ALIGN>
__global__ void __launch_bounds__(640, 1) k_fp4_wide(const __grid_constant__ Fp4MmParams p) {
    using S = Wide<FMT>;
    extern __shared__ uint8_t raw[];
    // full (codes), scaled, drained: the first CTA's count for both; landed
    // (scales), empty, sums: each CTA its own
    __shared__ __align__(8) uint64_t full[S::kStages], landed[S::kStages], empty[S::kStages];
    __shared__ __align__(8) uint64_t scaled[S::kSfBufs], sums, drained, done;
    __shared__ uint32_t tmem_at;
    __shared__ volatile int abort_flag;
    uint8_t *ring = raw + ((1024u - (dev::smem_addr(raw) & 1023u)) & 1023u);

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same for a warp
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
    }
    if (warp == 2 && lane == 0) {
        dev::prefetch_tensormap(&p.x);
        dev::prefetch_tensormap(&p.xs);
        dev::prefetch_tensormap(&p.w[GATED ? rank : 0]);
        dev::prefetch_tensormap(&p.ws[0]);
        if (GATED) dev::prefetch_tensormap(&p.ws[1]);
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
    if (warp == 0 && dev::elect_one()) {
        auto at = [&](int map) { return (p.moves >> map) & 1u ? w.e : 0; };
        bool dropped = false, ok = true;
        int i = 0;  // stages loaded
        Slot<S::kStages> s;
        while (ok && w.next()) {
            for (int k = 0; k < p.stages_k; ++k, ++i, s.next()) {
                const int st = s.at;
                if (i >= S::kStages && !dev::mbar_wait_bounded(&empty[st], s.parity ^ 1,
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
    } else if (warp == 1 && rank == 0 && dev::elect_one()) {
        constexpr uint32_t word = dev::mma_word(FMT, 256, 256);
        bool ok = true;
        int n = 0;  // tiles
        Slot<S::kStages> s;
        Slot<S::kSfBufs> f;
        bool ready = false;
        const uint64_t first = dev::operand_desc(dev::smem_addr(ring));
        for (; ok && w.next(); ++n) {
            if (n > 0 && !dev::mbar_wait_bounded(&drained, (n - 1) & 1, p.wait_limit_ns,
                                                 &abort_flag)) {
                gave_up();
                break;
            }
            const uint32_t d = tmem + (n & 1) * S::kOther;
            for (int k = 0; k < p.stages_k; ++k, s.next()) {
                const uint64_t xd = first + (uint32_t)(s.at * (S::kStage >> 4));
                const uint64_t wd = xd + (S::kCodes >> 4);
                const uint32_t sx = tmem + S::kScales + f.at * S::kSfCols;
                const uint32_t sw = sx + 4 * S::KT;
                const int steps = p.mma_k - 4 * k;  // 64-column steps left
                if (!ready && !dev::mbar_wait_bounded(&scaled[f.at], f.parity, p.wait_limit_ns,
                                                      &abort_flag)) {
                    gave_up();
                    ok = false;
                    break;
                }
                dev::tc_fence_after();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j >= steps) break;
                    const int t = j * S::KT / 4;
                    dev::mma_fp4<FMT, 2>(
                        d, xd + 2 * j, wd + 2 * j,
                        dev::mma_word_id(word, FMT == FP8BQ_MXFP4 ? 2 * (j & 1) : 0), sx + 4 * t,
                        sw + 8 * t, j > 0 || k > 0);
                }
                f.next();
                ready = dev::mbar_try_wait(&scaled[f.at], f.parity);  // the next stage's
                dev::mma_commit<2>(&empty[s.at]);
            }
            dev::mma_commit<2>(&sums);
        }
        dev::mma_commit_pair_here(&done);
        if (!dev::mbar_wait_bounded(&done, 0, kDrainNs, nullptr)) atomicOr(&g_fp4_error_word, 2u);
    } else if (warp >= 4 && (warp < 8 || warp >= 16)) {
        const int turn = warp >> 4;
        const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
        bool ok = true;
        Slot<S::kStages> s, old;  // `old`: kSfBufs stages behind
        Slot<S::kSfBufs> f;
        for (int i = 0; ok && w.next();) {
            for (int k = 0; k < p.stages_k; ++k, ++i, s.next(), f.next()) {
                if ((i & 1) != turn) {
                    if (i >= S::kSfBufs) old.next();
                    continue;
                }
                bool here = dev::mbar_wait_bounded(&landed[s.at], s.parity, p.wait_limit_ns,
                                                   &abort_flag);
                if (rank == 0)
                    here = here && dev::mbar_wait_bounded(&full[s.at], s.parity, p.wait_limit_ns,
                                                          &abort_flag);
                const uint8_t *sf = ring + s.at * S::kStage + 2 * S::kCodes + lane * 16;
                uint4 v[3 * S::KT];  // of the tokens, then tile by tile of the weight's two rows
#pragma unroll
                for (int t = 0; t < S::KT; ++t) {
                    v[t] = *(const uint4 *)(sf + t * kFp4TileBytes);
                    v[S::KT + 2 * t] = *(const uint4 *)(sf + S::SF + t * kFp4TileBytes);
                    v[S::KT + 2 * t + 1] = *(const uint4 *)(sf + 2 * S::SF + t * kFp4TileBytes);
                }
                if (i >= S::kSfBufs) {  // the products that read this buffer are done
                    here = here && dev::mbar_wait_bounded(&empty[old.at], old.parity,
                                                          p.wait_limit_ns, &abort_flag);
                    old.next();
                }
                if (!__all_sync(0xffffffffu, here)) {
                    if (lane == 0) gave_up();
                    ok = false;
                    break;
                }
                dev::tc_fence_after();
                scales_to_tmem<3 * S::KT>(tmem + quarter + S::kScales + f.at * S::kSfCols, v);
                dev::tc_fence_before();
                __syncwarp();
                if (lane == 0) dev::peer_arrive(dev::peer_addr(dev::smem_addr(&scaled[f.at]), 0));
            }
        }
    } else if (warp >= 8) {
        const int quarter = warp & 3, half = (warp - 8) >> 2;
        [[maybe_unused]] char *buf = (char *)ring + S::kStages * S::kStage + (warp - 8) * S::kStore;
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
            const int m0 = w.m0 + (int)rank * 128 + quarter * 32;  // the warp's first row
            [[maybe_unused]] const bool in = m0 + lane < w.valid;
            const float xt = MM_XT(p, w.e), alpha = __fmul_rn(xt, MM_WT(p, 0, w.e));
            const float alpha1 = GATED ? __fmul_rn(xt, MM_WT(p, 1, w.e)) : 0.0f;
            // Runs of 16 columns, every other one of them this warp's, from
            // the side whose columns the next tile shares: those (gated: the
            // up sums of even tiles, the gate's of odd ones) are all read
            // before anything is stored.
            constexpr int kRuns = GATED ? 4 : 8;
            const bool odd = n & 1;
            auto run = [&](int i) { return half + 2 * (odd ? i : kRuns - 1 - i); };
            const uint32_t shared = d + (GATED && !odd ? 128 : 0);
            const uint32_t others = d + (GATED && odd ? 128 : 0);
            uint32_t pre[3][16];
#pragma unroll
            for (int i = 0; i < 3; ++i) dev::tmem_ld16(shared + 16 * run(i), pre[i]);
            dev::tmem_ld_wait();
            dev::tc_fence_before();
            __syncwarp();
            if (lane == 0) dev::peer_arrive(drained_bar);
            auto store = [&](int i, const uint32_t (&x)[16], const uint32_t (&y)[16]) {
                float v[16];
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    if constexpr (GATED) {
                        const float g = __uint_as_float(odd ? x[q] : y[q]);
                        const float u = __uint_as_float(odd ? y[q] : x[q]);
                        v[q] = silu<BF16>(g * alpha) * (u * alpha1);
                    } else {
                        v[q] = __uint_as_float(x[q]) * alpha;
                    }
                }
                const int c = w.n0 + 16 * run(i);
                if constexpr (fp4_staged(ALIGN, BF16 ? 2 : 4)) {
                    if (c < p.N) store16_staged<BF16, ALIGN>(p, w.e, m0, w.valid - m0, c, v, buf, lane);
                } else if (in && c < p.N) {
                    store16<BF16>(p, w.e, m0 + lane, c, v);
                }
            };
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                uint32_t y[16];
                if constexpr (GATED) {
                    dev::tmem_ld16(others + 16 * run(i), y);
                    dev::tmem_ld_wait();
                }
                store(i, pre[i], GATED ? y : pre[i]);
            }
#pragma unroll 1
            for (int i = 3; i < kRuns; ++i) {
                uint32_t x[16], y[16];
                dev::tmem_ld16(shared + 16 * run(i), x);
                if constexpr (GATED) dev::tmem_ld16(others + 16 * run(i), y);
                dev::tmem_ld_wait();
                store(i, x, GATED ? y : x);
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
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                cudaSharedmemCarveoutMaxShared);
}

template <typename K>
cudaError_t launch_clusters(K kern, dim3 grid, unsigned threads, unsigned cluster, int smem,
                            cudaStream_t st, const Fp4MmParams &p) {
    g_fp4_launched.store(true, std::memory_order_relaxed);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    if (cluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = cluster;
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    if (p.overlap) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// Clusters of each size that fit on the device at once (a size that the device
// cannot run counts as 0).
constexpr int kSplits[] = {2, 3, 4, 6, 8};  // 5 and 7 measured no better than 4 and 6
struct ClusterFit {
    cudaError_t attr = cudaSuccess;
    int n[9] = {};
};

// The occupancy calls count one CTA an SM for any kernel that allocates tensor
// memory; `per_sm` CTAs are resident (1187 tiles of 128 outputs, one token, K
// = 4096: 56.5 us with 296 persistent CTAs, 75.5 with 148).
template <typename K>
ClusterFit cluster_fit(K kern, unsigned threads, int smem, int per_sm) {
    ClusterFit f;
    f.attr = set_smem(kern, smem);
    auto ask = [&](int c) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = 8 * c;
        cfg.blockDim = threads;
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = c;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&f.n[c], kern, &cfg);
        if (e != cudaSuccess) {
            f.n[c] = 0;
            // any other failure is the call's: with fewer clusters it would add up
            // other parts
            if (c == 1 || (e != cudaErrorInvalidClusterSize && e != cudaErrorInvalidConfiguration))
                f.attr = e;
            else
                cudaGetLastError();
        }
        f.n[c] *= per_sm;
    };
    if (f.attr == cudaSuccess) ask(1);
    for (int c : kSplits)
        if (f.attr == cudaSuccess) ask(c);
    if (f.attr == cudaSuccess && f.n[1] < 1) f.attr = cudaErrorInvalidConfiguration;
    return f;
}

template <int FMT, bool GATED, bool BF16, int NT>
cudaError_t narrow(const Fp4MmParams &p0, cudaStream_t st) {
    using S = Narrow<FMT, GATED, NT>;
    auto kern = k_fp4_narrow<FMT, GATED, BF16, NT>;
    static PerDevice<ClusterFit> setup;
    const ClusterFit fit =
        setup.get([&] { return cluster_fit(kern, S::kThreads, S::kSmem, S::kTwo ? 2 : 1); },
                  [](const ClusterFit &f) { return f.attr == cudaSuccess; });
    if (fit.attr != cudaSuccess) return fit.attr;
    Fp4MmParams p = p0;
    const int64_t tiles = (int64_t)((p.N + 127) / 128) * ((p.M + NT - 1) / NT) * p.batch;
    // The largest of these cluster sizes with which every tile runs at once
    // and each CTA has a stage.
    p.split = 1;
    for (int c : kSplits)
        if (tiles <= fit.n[c] && c <= p.stages_k) p.split = c;
    const int64_t clusters = p.split > 1 || tiles < fit.n[1] ? tiles : fit.n[1];
    return launch_clusters(kern, dim3((unsigned)(clusters * p.split)), S::kThreads,
                           (unsigned)p.split, S::kSmem, st, p);
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

template <int FMT, bool GATED, bool BF16, int ALIGN>
cudaError_t wide(const Fp4MmParams &p, cudaStream_t st) {
    using S = Wide<FMT>;
    auto kern = k_fp4_wide<FMT, GATED, BF16, ALIGN>;
    static PerDevice<cudaError_t> setup;
    const cudaError_t e = setup.get([&] { return set_smem(kern, S::kSmem); },
                                    [](cudaError_t r) { return r == cudaSuccess; });
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)((p.M + 255) / 256) * ((p.N + (GATED ? 127 : 255)) / (GATED ? 128 : 256)) *
                          p.batch;
    const int64_t pairs = sm_count() / 2;
    return launch_clusters(kern, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), S::kThreads, 2,
                           S::kSmem, st, p);
}

template <int FMT, bool GATED, bool BF16>
cudaError_t wide_store(const Fp4MmParams &p, cudaStream_t st) {
    if (!BF16 && p.store_align >= 32) return wide<FMT, GATED, BF16, BF16 ? 16 : 32>(p, st);
    if (p.store_align >= 16) return wide<FMT, GATED, BF16, 16>(p, st);
    if (!BF16 || p.store_align >= 4) return wide<FMT, GATED, BF16, 4>(p, st);
    return wide<FMT, GATED, BF16, BF16 ? 2 : 4>(p, st);
}

template <int FMT>
cudaError_t wide_format(const Fp4MmParams &p, bool gated, bool bf16, cudaStream_t st) {
    if (gated) return bf16 ? wide_store<FMT, true, true>(p, st) : wide_store<FMT, true, false>(p, st);
    return bf16 ? wide_store<FMT, false, true>(p, st) : wide_store<FMT, false, false>(p, st);
}

}  // namespace

cudaError_t launch_fp4_mm_wide(const Fp4MmParams &p, int format, bool gated, bool out_bf16,
                               cudaStream_t st) {
    return format == FP8BQ_MXFP4 ? wide_format<FP8BQ_MXFP4>(p, gated, out_bf16, st)
                                 : wide_format<FP8BQ_NVFP4>(p, gated, out_bf16, st);
}

// The kernel for a product, and what it takes about: the tile's width in
// tokens of the few-token kernel, or 0 for the many-token one.  Up to 32 tokens
// the narrowest tile that holds them; beyond, the one with the shortest
// estimate.  A call takes about
//     begin + stage * (stages of a CTA)
//           + max(again * (stages), round) * (rounds - 1)
// microseconds, rounds = tiles over the tiles that run at once; `round` is the
// time to store a tile, and `staged` what a round of the many-token kernel
// takes longer where its outputs pass through shared memory.  Fitted to B200,
// 1000 x 4100 to 12288 x 4096 and 4096 x 12288, stacks of 8 to 128 of 768 x 2048
// to 4096 x 4096, 40 to 8192 tokens, mxfp4: the choice costs 1 to 2 % of the best
// one's time on average (measured, us, many-token / 64 / 128 / 256 wide tiles):
//     515 tokens, 1000 x 4100    13.0 / 10.2 /  9.3 / 11.3
//     1500 tokens, 1001 x 700     8.7 /  5.5 /  5.6 /  9.2
//     8192 tokens, 6148 x 512    46.1 / 52.5 / 61.3 / 61.5
//     256 tokens, 4096 x 4096     9.9 /  9.6 /  8.7 / 10.5
//     256 tokens, 12288 x 4096   10.5 / 16.2 / 15.3 / 15.5
//     300 tokens, 4096 x 12288   19.3 / 20.7 / 19.0 / 16.7
//     1024 tokens, 6144 x 4096   16.5 / 22.5 / 19.8 / 23.0
//     gated, 256 x 4096 x 4096   10.6 / 10.8 / 11.7
//     gated, 64 x 12288 x 4096   15.9 / 10.9 / 11.5
//     128 of 128 x 2048 x 768    41.0 / 39.0 / 41.0 / 51.1
int fp4_choose(int64_t M, int64_t N, int64_t stages, int64_t batch, bool gated, bool staged,
               double *us) {
    struct Cost {
        int tokens;
        double begin, stage, again, round, staged;
    };
    static constexpr Cost plain[] = {{16, 4.5, 0.33, 0.40, 2.5, 0},  {32, 4.9, 0.33, 0.42, 2.1, 0},
                                     {0, 5.7, 0.28, 0.43, 2.1, 2.0}, {64, 6.3, 0.34, 0.43, 2.1, 0},
                                     {128, 6.2, 0.24, 0.36, 2.4, 0}, {256, 8.2, 0.28, 0.61, 5.2, 0}};
    static constexpr Cost both[] = {{16, 5.1, 0.45, 0.60, 2.6, 0},  {32, 6.1, 0.45, 0.60, 2.6, 0},
                                    {0, 5.9, 0.30, 0.43, 2.7, 1.5}, {64, 6.5, 0.30, 0.43, 2.35, 0},
                                    {128, 8.6, 0.34, 0.73, 4.2, 0}};
    const double sms = sm_count();
    const int first = M <= 16 ? 0 : M <= 32 ? 1 : 2, last = M <= 32 ? first : gated ? 4 : 5;
    int best = 0;
    for (int i = first; i <= last; ++i) {
        const Cost &c = gated ? both[i] : plain[i];
        const int64_t rows = c.tokens ? c.tokens : 256, cols = c.tokens || gated ? 128 : 256;
        const double tiles = (double)((M + rows - 1) / rows) * (double)((N + cols - 1) / cols) * batch;
        const bool two = c.tokens && c.tokens <= (gated ? 16 : 64);  // CTAs an SM
        const double once = c.tokens == 0 ? sms / 2 : two ? 2 * sms : sms;
        double share = (double)stages;  // stages of a CTA where a cluster splits K
        if (c.tokens)
            for (int s : kSplits)  // clusters of more than two leave some SMs out
                if (s <= stages && tiles * s <= once * (s == 2 ? 1.0 : s == 8 ? 0.82 : 0.9))
                    share = (double)((stages + s - 1) / s);
        const double rounds = (double)(int64_t)((tiles + once - 1) / once);
        const double again = c.again * stages > c.round ? c.again * stages : c.round;
        const double t = c.begin + c.stage * share + again * (rounds - 1) +
                         (staged ? c.staged * rounds : 0);
        if (i == first || t < *us) {
            *us = t;
            best = c.tokens;
        }
    }
    return best;
}

cudaError_t launch_fp4_mm_narrow(const Fp4MmParams &p, int format, bool gated, bool out_bf16,
                                 int tokens, cudaStream_t st) {
    return format == FP8BQ_MXFP4 ? narrow_format<FP8BQ_MXFP4>(p, gated, out_bf16, tokens, st)
                                 : narrow_format<FP8BQ_NVFP4>(p, gated, out_bf16, tokens, st);
}

cudaError_t read_and_clear_fp4_error_word(uint32_t *out) {
    *out = 0;
    if (!g_fp4_launched.load(std::memory_order_relaxed)) return cudaSuccess;
    uint32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_fp4_error_word, sizeof(uint32_t));
    if (e != cudaSuccess) return e;
    if (*out) e = cudaMemcpyToSymbol(g_fp4_error_word, &zero, sizeof(uint32_t));
    return e;
}

FP8BQ_DEFINE_BOUNDS_RECORD(bounds_record_fp4_mm)

}  // namespace fp8bq
