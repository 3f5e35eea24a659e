// GEMM on 8-bit rows on the 5th-generation tensor cores: out[M,N] = (xq xs)(wq ws)^T, e4m3
// operands with one fp32 scale per row of x and per row of w, fp32 accumulation in tensor memory.
// The scales do not depend on k, so the product of the codes is scaled once, in the epilogue, by the row's
// scale and then by the column's (RowScale).
//
// What each has to do: M N K products of codes and, once each, K (M + N) bytes of codes and the
// outputs.  Many rows are bound by the tensor cores (and, past a hundred microseconds, by the power they
// may draw), few rows by the launch, the loads' latency and what a k-block costs to issue.
//
// Two forms with the roles of the bf16 GEMM: one warp issues TMA loads of 128 k-bytes (128-byte
// swizzle) into a ring, one issues tcgen05.mma kind::f8f6f4 into one of two accumulators, the others drain
// the other accumulator.  The issuing warps run their loops whole and one elected lane issues: with one
// lane alone in the loop an MMA took 68 clocks to issue, a commit 61, a k-block 530 whatever its tile -- more
// than the 512 of a pair's products.  Elected, an MMA takes 24 and a k-block 300 (23,460 x 6144 x 1024: 99.7 ->
// 86.7 us).
//   k_gemm_q8_pair: persistent over tiles of 256 x 256 by pairs of CTAs (cta_group::2).  Each CTA holds
// 128 rows of x and 128 rows of w of a k-block, 32 KB, and the pair's tensor cores read both halves of w; a
// 128 x 256 tile of one CTA would load 48 KB for the same products, more than the 64 bytes a clock
// that an SM takes from L2 (such tiles ran at 2,770 TFLOP/s, what that rate allows).  Outputs
// leave as TMA tiles of 32 rows: fp32 columns as they are, the residual as reducing stores
// (each element is added to once, so the sum's bits do not depend on order; a subnormal sum may become
// zero), SwiGLU pairs as bf16.  With SwiGLU 23,460 x 6144 x 1024 takes 86 us, 3,420 TFLOP/s, in bursts of some 40
// launches, and 101 when it runs on and on; 8,191 x 7,168 x 8,192 to fp32 276 us, 3,490 TFLOP/s, and 319, at the power
// limit (1,390 MHz).  23,460 x 1024 x 2048 with the residual, bound by bytes, 50.6 (floor 36.3).
// Sharing the rows of x between two pairs by TMA multicast made mid sizes up to 8% faster and the
// large ones up to 5% slower, and is not done.
//   k_gemm_q8: tiles of 128 x BN by single CTAs, for few rows or few tiles: persistent, or, with fewer
// tiles than SMs and a long K, a cluster of 2 to 8 CTAs to a tile, each with a share of K; the shares meet
// in distributed shared memory in a fixed order.  33 x 1024 x 2048 with the residual: 4.0 us; 128 x 4096 x 4096 6.8
// (floor 2.9).  Between 200 and 4,096 rows both forms are 1.8 to 4.5 times their floor (2,048 x 6144 x 1024 11.9 us, 600
// rows 7.2): a pair's first and last tile outside the products, rounds that are partly filled, rows stored by lanes.
// M, N and K need not fill tiles: TMA zero-fills past the tensors' ends (a zero code adds
// nothing) and drops what is stored past them; N and K are multiples of 16.
// Every mbarrier wait is bounded.  A role that gives up stops; the epilogue then gives up too, and what it had not
// finished is NaN in the outputs.  No CTA leaves, or reuses its ring, before the copies it issued have landed and the
// MMAs have completed.

#include "kernels.h"
#include "tc.cuh"

namespace q3 {

namespace {

constexpr int G8_BM = 128, G8_BK = 128;  // BK in bytes = e4m3 elements
constexpr int G8_THREADS = 320, G8_EPI_WARPS = 8;
constexpr int MAX_SPLIT = 8;  // CTAs that may share a tile's K

// ---- tiles of one CTA ---------------------------------------------------------------------

template <int BN>
struct G8 {
    static constexpr int A_BYTES = G8_BM * G8_BK, B_BYTES = BN * G8_BK;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = BN >= 128 ? 6 : BN >= 64 ? 8 : 10;
    static constexpr int SMEM = STAGES * STAGE + 256 + 1024;  // ring + barriers + alignment
    static constexpr int PITCH = (BN + 4) * 4;  // bytes of a row of sums in shared memory, 4 banks past the last row's
    static constexpr int SCALES = G8_BM * PITCH;   // the rows' scales, behind the sums
    static_assert(SCALES + G8_BM * 8 <= STAGES * STAGE, "sums and scales exceed the ring");
    static constexpr uint32_t TMEM_COLS = 2 * BN < 32 ? 32 : 2 * BN;
};

// Instruction descriptor of kind::f8f6f4: fp32 accumulator, e4m3 A and B (format 0), both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
constexpr uint32_t NAN_BITS = 0x7fffffffu;
// Place in a ring of N stages and the parity of the round there.
template <int N>
struct Ring {
    uint32_t s = 0, round = 0;
    __device__ __forceinline__ void next() {
        if (++s == N) {
            s = 0;
            round ^= 1;
        }
    }
};

// The products of one k-block: x and w at these shared addresses, 32 k-bytes an instruction.
template <int CTAS>
__device__ __forceinline__ void mma_block(uint32_t acc, uint32_t sa, uint32_t sb, uint32_t idesc, uint32_t accumulate) {
    const uint64_t a = sdesc_k_sw128(sa), b = sdesc_k_sw128(sb);
#pragma unroll
    for (int k = 0; k < G8_BK / 32; ++k)
        if (CTAS == 2)
            asm volatile(
                "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(acc),
                "l"(a + 2 * k), "l"(b + 2 * k), "r"(idesc), "r"(k ? 1u : accumulate));
        else
            asm volatile(
                "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(acc),
                "l"(a + 2 * k), "l"(b + 2 * k), "r"(idesc), "r"(k ? 1u : accumulate));
}

__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Shared address of the same place in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(p), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t in_cta(const void *p, uint32_t rank) { return in_cta(smem_addr(p), rank); }
__device__ __forceinline__ float4 load_from(uint32_t addr) {  // shared memory of the cluster
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// A row's scale as s f, f a power of two and 1 for any usual row: outputs are ((sum s) w) f.  The codes' sum is 0 or
// 2^-18 to 2^48, so that its product with s is a normal number, and that product times w leaves fp32 only where
// the output does.  (The two scales' product formed first may be zero, or infinite and with a zero sum NaN.)
struct RowScale {
    float s, f;
    RowScale() = default;
    __device__ __forceinline__ explicit RowScale(float scale) {
        const float m = fabsf(scale);
        f = m > 0x1p78f ? 0x1p56f : m < 0x1p-104f && m > 0.0f ? 0x1p-44f : 1.0f;
        s = scale * (m > 0x1p78f ? 0x1p-56f : m < 0x1p-104f ? 0x1p44f : 1.0f);
    }
    __device__ __forceinline__ float times(float sum, float w) const { return sum * s * w * f; }
};

// 16 columns of one output row: what they need besides the accumulator, and their store.
template <int EPI>
struct Out16 {
    float4 w[4], r[EPI == EPI_RESID_ADD ? 4 : 1];

    // Column scales, and the residual of a row (out of this row and these columns), read while the
    // MMAs run: at 33 rows the residual's latency was a tenth of the launch.
    __device__ __forceinline__ void read(const float *ws, const void *out, size_t row, int col, int N, bool live) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = __ldg(reinterpret_cast<const float4 *>(ws + col) + j);
            if (EPI == EPI_RESID_ADD && live)
                r[j] = *(reinterpret_cast<const float4 *>(static_cast<const float *>(out) + row * N + col) + j);
        }
    }
    __device__ __forceinline__ void store(const uint32_t *v, const RowScale &sx, size_t row, int col, int N,
                                          void *out) const {
        float y[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[4 * j] = sx.times(__uint_as_float(v[4 * j]), w[j].x);
            y[4 * j + 1] = sx.times(__uint_as_float(v[4 * j + 1]), w[j].y);
            y[4 * j + 2] = sx.times(__uint_as_float(v[4 * j + 2]), w[j].z);
            y[4 * j + 3] = sx.times(__uint_as_float(v[4 * j + 3]), w[j].w);
        }
        if (EPI == EPI_SWIGLU) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[j] = pack_bf16x2(swiglu(y[4 * j], y[4 * j + 1]), swiglu(y[4 * j + 2], y[4 * j + 3]));
            *reinterpret_cast<uint4 *>(static_cast<bf16 *>(out) + row * (N / 2) + col / 2) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
            float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(out) + row * N + col);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float4 t = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
                if (EPI == EPI_RESID_ADD) {
                    t.x += r[j].x;
                    t.y += r[j].y;
                    t.z += r[j].z;
                    t.w += r[j].w;
                }
                dst[j] = t;
            }
        }
    }
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}

// What an epilogue warp's wait that gave up leaves: NaN in row r and the warp's columns of tile t and of the CTA's tiles
// after it.  A call, so that its code is not in the way of ordinary launches.
template <int BN, int EPI>
__device__ __noinline__ void store_nan(long long t, long long tiles, long long step, int tiles_n, int r, int half, int M, int N,
                                       void *out) {
    for (; t < tiles; t += step) {
        const int row = (int)(t / tiles_n) * G8_BM + r, n0 = (int)(t % tiles_n) * BN;
        for (int c = half; c < BN / 16; c += 2)
            for (int col = n0 + c * 16; row < M && col < min(N, n0 + c * 16 + 16); ++col)
                if (EPI != EPI_SWIGLU)
                    static_cast<float *>(out)[(size_t)row * N + col] = __uint_as_float(NAN_BITS);
                else if (col % 2 == 0)
                    static_cast<uint16_t *>(out)[(size_t)row * (N / 2) + col / 2] = 0x7fff;
    }
}

// Rows of x in a box: 128, or all there are in whole swizzle groups (16 rows of x against
// 4096 x 4096 weights: 14.4 us with boxes of 128 rows, mostly zero fill, 10.8 with 16).
__host__ __device__ constexpr uint32_t q8_box_rows(int M) { return M >= 128 ? 128 : (M + 7) / 8 * 8; }

template <int BN, int EPI, bool SPLIT>
__global__ void __launch_bounds__(G8_THREADS, 1) k_gemm_q8(const __grid_constant__ CUtensorMap tmA,
                                                           const __grid_constant__ CUtensorMap tmB,
                                                           const float *__restrict__ xs, const float *__restrict__ ws, int M,
                                                           int N, int K, void *out, int S, long long limit) {
    using T = G8<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + T::STAGES * T::STAGE);
    uint64_t *empty = full + T::STAGES;
    uint64_t *tm_full = empty + T::STAGES;  // [2]
    uint64_t *tm_empty = tm_full + 2;       // [2]
    uint64_t *drained = tm_empty + 2;       // the MMAs issued, where a wait gave up
    uint64_t *idle = drained + 1;           // no copy and no MMA is in flight
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(idle + 1);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    // this CTA's k-blocks: all, or its share of the cluster's tile
    const int KB_ALL = (K + G8_BK - 1) / G8_BK, rank = SPLIT ? (int)cta_rank() : 0;
    const int kb0 = SPLIT ? KB_ALL * rank / S : 0, KB = (SPLIT ? KB_ALL * (rank + 1) / S : KB_ALL) - kb0;
    // With fewer than 128 rows of x only theirs are loaded: the rest of the tile holds whatever
    // shared memory held, and its products, in rows of their own, are not stored.
    const uint32_t stage_bytes = q8_box_rows(M) * G8_BK + T::B_BYTES;
    const int tiles_n = (N + BN - 1) / BN;
    const long long tiles = (long long)((M + G8_BM - 1) / G8_BM) * tiles_n;
    const long long first = SPLIT ? blockIdx.x / S : blockIdx.x, step = SPLIT ? tiles : gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < T::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tm_full[a], 1);
            mbar_init(&tm_empty[a], G8_EPI_WARPS);  // one arrival per epilogue warp
        }
        mbar_init(drained, 1);
        mbar_init(idle, 2);  // the warps that issue
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(T::TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    pdl_wait();
    pdl_trigger();

    if (warp == 0) {
        const bool issues = elect_one();
        Ring<T::STAGES> r;
        uint32_t it = 0;  // k-blocks issued so far
        bool ok = true;
        for (long long t = first; t < tiles && ok; t += step) {
            const int m0 = (int)(t / tiles_n) * G8_BM, n0 = (int)(t % tiles_n) * BN;
            for (int kb = 0; kb < KB; ++kb, ++it, r.next()) {
                if (it >= T::STAGES && !warp_wait(&empty[r.s], r.round ^ 1, limit)) {
                    ok = false;
                    break;
                }
                uint8_t *sa = smem + r.s * T::STAGE;
                if (issues) {
                    mbar_expect_tx(&full[r.s], stage_bytes);
                    tma_load_2d(sa, &tmA, (kb0 + kb) * G8_BK, m0, &full[r.s]);
                    tma_load_2d(sa + T::A_BYTES, &tmB, (kb0 + kb) * G8_BK, n0, &full[r.s]);
                }
            }
        }
        // the ring's last copies land before the CTA can leave, whether or not their MMAs are issued
#pragma unroll 1
        for (uint32_t s = 0; s < (it < T::STAGES ? it : T::STAGES); ++s)
            warp_wait(&full[s], s < r.s ? r.round : r.round ^ 1, WAIT_LIMIT_DEFAULT);
        if (SPLIT && issues) mbar_arrive_cta(idle);
    } else if (warp == 1) {
        constexpr uint32_t idesc = idesc_e4m3(G8_BM, BN);
        const bool issues = elect_one();
        Ring<T::STAGES> r;
        uint32_t local = 0;
        bool ok = true;
        for (long long t = first; t < tiles && ok; t += step, ++local) {
            const uint32_t a = local & 1;
            if (local >= 2 && !warp_wait(&tm_empty[a], ((local >> 1) & 1) ^ 1, limit)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + a * BN;
            for (int kb = 0; kb < KB; ++kb, r.next()) {
                if (!warp_wait(&full[r.s], r.round, limit)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = smem_addr(smem + r.s * T::STAGE);
                if (issues) {
                    mma_block<1>(acc, sa, sa + T::A_BYTES, idesc, kb);
                    tc_commit(&empty[r.s]);
                }
            }
            if (ok && issues) tc_commit(&tm_full[a]);
        }
        __syncwarp();
        // the MMAs complete before the CTA can leave, whether or not the epilogue waits for them
        if (!ok && issues) tc_commit(drained);
        warp_wait(ok ? &tm_full[(local - 1) & 1] : drained, ok ? ((local - 1) >> 1) & 1 : 0, WAIT_LIMIT_DEFAULT);
        if (SPLIT && issues) mbar_arrive_cta(idle);
    } else {
        const int q = warp & 3;            // TMEM lane quarter this warp may access
        const int half = (warp - 2) >> 2;  // 16-column chunks half, half + 2, ... of the tile
        uint32_t local = 0;
        for (long long t = first; t < tiles; t += step, ++local) {
            const uint32_t a = local & 1;
            const int m0 = (int)(t / tiles_n) * G8_BM, n0 = (int)(t % tiles_n) * BN;
            const int row = m0 + q * 32 + lane;
            const bool live = row < M;
            const RowScale sx(live ? xs[row] : 0.0f);
            if (SPLIT) {  // its sums into shared memory, over the ring that the MMAs are done with
                const bool done = warp_poll(&tm_full[a], 0, limit);
                if (!done) warp_wait(idle, 0, WAIT_LIMIT_DEFAULT);
                tc_fence_after();
                float4 *dst = reinterpret_cast<float4 *>(smem + (q * 32 + lane) * T::PITCH);
                if (half == 0 && live) *reinterpret_cast<RowScale *>(smem + T::SCALES + (q * 32 + lane) * 8) = sx;
#pragma unroll
                for (int c = half; c < BN / 16; c += 2) {
                    uint32_t v[16];
                    tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + c * 16, v);
                    if (!done)  // a wait gave up: the outputs say so
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = NAN_BITS;
                    if (live)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            dst[c * 4 + j] = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                                         __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
                }
                break;
            }
            Out16<EPI> o;
            if (n0 + half * 16 < N) o.read(ws, out, row, n0 + half * 16, N, live);
            if (!warp_poll(&tm_full[a], (local >> 1) & 1, limit)) {  // NaN in this tile and in those after it
                store_nan<BN, EPI>(t, tiles, step, tiles_n, q * 32 + lane, half, M, N, out);
                break;
            }
            tc_fence_after();
            const uint32_t t_row = tmem + a * BN + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
            for (int c = half; c < BN / 16; c += 2) {
                const int col = n0 + c * 16;
                if (col >= N) break;
                uint32_t v[16];
                tmem_ld16(t_row + c * 16, v);
                if (live) o.store(v, sx, row, col, N, out);
                if (c + 2 < BN / 16 && col + 32 < N) o.read(ws, out, row, col + 32, N, live);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cta(&tm_empty[a]);
        }
    }
    tc_fence_before();
    if (SPLIT) {
        // Every CTA finishes a part of the tile: the shares of K in their order, a piece of 4 columns
        // (8 for SwiGLU) to a thread.
        __syncwarp();
        cluster_sync();  // the shares are in shared memory
        if (warp >= 2) {
            constexpr int W = EPI == EPI_SWIGLU ? 8 : 4, PIECES = BN / W;
            const int m0 = (int)(first / tiles_n) * G8_BM, n0 = (int)(first % tiles_n) * BN;
            const int rows = M - m0 < G8_BM ? M - m0 : G8_BM;
            for (int i = rank * (G8_EPI_WARPS * 32) + (int)threadIdx.x - 64; i < rows * PIECES; i += S * G8_EPI_WARPS * 32) {
                const int r = i / PIECES, c = i % PIECES * W, col = n0 + c;
                if (col >= N) continue;
                const uint32_t mine = smem_addr(smem + r * T::PITCH + c * 4);
                float4 part[W / 4][MAX_SPLIT];
#pragma unroll
                for (int j = 0; j < MAX_SPLIT; ++j)
                    if (j < S)
#pragma unroll
                        for (int h = 0; h < W / 4; ++h) part[h][j] = load_from(in_cta(mine + h * 16, j));
                const RowScale sx = *reinterpret_cast<const RowScale *>(smem + T::SCALES + r * 8);
                float y[W];
#pragma unroll
                for (int h = 0; h < W / 4; ++h) {
                    float4 v = part[h][0];
#pragma unroll
                    for (int j = 1; j < MAX_SPLIT; ++j)
                        if (j < S) {
                            v.x += part[h][j].x;
                            v.y += part[h][j].y;
                            v.z += part[h][j].z;
                            v.w += part[h][j].w;
                        }
                    const float4 w = __ldg(reinterpret_cast<const float4 *>(ws + col) + h);
                    y[4 * h] = sx.times(v.x, w.x);
                    y[4 * h + 1] = sx.times(v.y, w.y);
                    y[4 * h + 2] = sx.times(v.z, w.z);
                    y[4 * h + 3] = sx.times(v.w, w.w);
                }
                if (EPI == EPI_SWIGLU) {
                    uint2 o;
                    o.x = pack_bf16x2(swiglu(y[0], y[1]), swiglu(y[2], y[3]));
                    o.y = pack_bf16x2(swiglu(y[W - 4], y[W - 3]), swiglu(y[W - 2], y[W - 1]));
                    *reinterpret_cast<uint2 *>(static_cast<bf16 *>(out) + (size_t)(m0 + r) * (N / 2) + col / 2) = o;
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(out) + (size_t)(m0 + r) * N + col);
                    float4 t = make_float4(y[0], y[1], y[2], y[3]);
                    if (EPI == EPI_RESID_ADD) {
                        const float4 h = *dst;
                        t.x += h.x;
                        t.y += h.y;
                        t.z += h.z;
                        t.w += h.w;
                    }
                    *dst = t;
                }
            }
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while another reads its shares
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(T::TMEM_COLS));
    }
}

// 2-D map of row-major codes [rows, cols] read as boxes of 128 columns x box_rows rows.
bool make_map_q8(CUtensorMap *map, const uint8_t *base, int rows, int cols, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)cols};
    const cuuint32_t box[2] = {(cuuint32_t)G8_BK, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---- tiles of a pair of CTAs --------------------------------------------------------------

constexpr int P8_BM = 256, P8_BN = 256;
constexpr int P8_HALF = 128 * G8_BK;        // 16 KB: a CTA's rows of x, or of w, of a k-block
constexpr int P8_STAGE = 2 * P8_HALF, P8_STAGES = 6;
// 16 epilogue warps of 64 columns each, with output tiles of 2 KB that leave room for a sixth stage: 8,191 x
// 7,168 x 8,192 290 -> 287 us, 23,460 x 4,096 x 1,024 to fp32 91 -> 88 against 8 warps, 4 KB and five.
constexpr int P8_EPI_WARPS = 16, P8_THREADS = 64 + P8_EPI_WARPS * 32;
constexpr int P8_TILE = 32 * 64;              // a warp's output tile: 32 rows of 64 bytes
constexpr int P8_OUT = P8_STAGES * P8_STAGE;  // the output tiles
constexpr int P8_BARS = P8_OUT + P8_EPI_WARPS * P8_TILE;
constexpr int P8_SMEM = P8_BARS + 256 + 1024;
static_assert(P8_SMEM <= 227 * 1024, "ring and output tiles exceed shared memory");

// TMA load into this CTA that completes on a barrier of either CTA.
__device__ __forceinline__ void tma_load_pair(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
        "[%1, {%3, %4}], [%2];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
// Arrives at this barrier's place in both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// Arrives on a barrier of either CTA; relaxed, since what it orders is the accumulator's reads, which
// tcgen05.wait::ld and the fence before it have completed (a release waits for this warp's stores): the PTX ISA's own
// pattern between threads for tcgen05 (wait, fence::before_thread_sync, relaxed arrival; wait, fence::after_thread_sync).
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A word of either CTA's shared memory.
__device__ __forceinline__ void store_to(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Takes `bytes` that will not come off what a barrier of this CTA expects.
__device__ __forceinline__ void complete_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}
// A shared tile to the output: stored, or added to it.  The caller commits the group.
template <bool ADD>
__device__ __forceinline__ void tile_out(const CUtensorMap *map, const void *src, int x, int y) {
    if (ADD)
        asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"(smem_addr(src)), "r"(x), "r"(y)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"(smem_addr(src)), "r"(x), "r"(y)
                     : "memory");
}
// Two products at once.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t x, y, z;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(z) : "l"(x), "l"(y));
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(z));
    return r;
}

template <int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(P8_THREADS, 1)
    k_gemm_q8_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmO, const float *__restrict__ xs, const float *__restrict__ ws,
                   int M, int N, int K, long long limit) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + P8_BARS);  // [stages], those of CTA 0 in use
    uint64_t *empty = full + P8_STAGES;                             // [stages]
    uint64_t *tm_full = empty + P8_STAGES;                          // [2]
    uint64_t *tm_empty = tm_full + 2;                               // [2], those of CTA 0 in use
    uint64_t *drained = tm_empty + 2;                               // all MMAs, at the end
    uint64_t *met = drained + 1;                                    // CTA 1 has issued its last load; CTA 0's in use
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(met + 1);
    uint32_t *issued1 = tmem_slot + 1;  // k-blocks that CTA 1 issued, then

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();
    const int KB = (K + G8_BK - 1) / G8_BK;
    const int tiles_n = (N + P8_BN - 1) / P8_BN;
    const long long tiles = (long long)((M + P8_BM - 1) / P8_BM) * tiles_n;
    const long long first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < P8_STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tm_full[a], 1);
            mbar_init(&tm_empty[a], 2 * P8_EPI_WARPS);  // one arrival per epilogue warp of the pair
        }
        mbar_init(drained, 1);
        mbar_init(met, 1);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(tmem_slot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are ready
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    pdl_wait();
    pdl_trigger();

    if (warp == 0) {
        const bool issues = elect_one();
        Ring<P8_STAGES> r;
        uint32_t it = 0;  // k-blocks issued so far
        bool ok = true;
        for (long long t = first; t < tiles && ok; t += step) {
            const int m0 = (int)(t / tiles_n) * P8_BM + (int)rank * 128;
            const int n0 = (int)(t % tiles_n) * P8_BN + (int)rank * 128;
            for (int kb = 0; kb < KB; ++kb, ++it, r.next()) {
                if (it >= P8_STAGES && !warp_wait(&empty[r.s], r.round ^ 1, limit)) {
                    ok = false;
                    break;
                }
                uint8_t *sa = smem + r.s * P8_STAGE;
                const uint32_t bar = in_cta(&full[r.s], 0);
                if (issues) {
                    if (rank == 0) mbar_expect_tx(&full[r.s], 2 * P8_STAGE);  // the bytes of both CTAs
                    tma_load_pair(sa, &tmA, kb * G8_BK, m0, bar);
                    tma_load_pair(sa + P8_HALF, &tmB, kb * G8_BK, n0, bar);
                }
            }
        }
        // The ring's last loads land before a CTA can leave, whether or not their MMAs are issued: CTA 0 waits for both
        // CTAs' bytes.  Where a wait gave up, one may have issued up to a ring more k-blocks than the other, and
        // CTA 0 makes its barriers whole first.
        if (rank == 1) {
            if (issues) {
                store_to(in_cta(issued1, 0), it);
                asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_cta(met, 0)) : "memory");
            }
        } else {
            const bool here = warp_wait(met, 0, WAIT_LIMIT_DEFAULT);
            asm volatile("fence.acq_rel.cluster;" ::: "memory");
            const uint32_t other = here ? *static_cast<volatile uint32_t *>(issued1) : it, most = it > other ? it : other;
            if (it != other && issues)
                for (uint32_t j = it < other ? it : other; j < most; ++j) {
                    if (it < other)
                        mbar_expect_tx(&full[j % P8_STAGES], P8_STAGE);  // CTA 1's bytes alone
                    else
                        complete_tx(&full[j % P8_STAGES], P8_STAGE);  // CTA 1's will not come
                }
            __syncwarp();
            for (uint32_t j = (most > P8_STAGES ? most - P8_STAGES : 0); j < most; ++j)
                warp_wait(&full[j % P8_STAGES], (j / P8_STAGES) & 1, WAIT_LIMIT_DEFAULT);
        }
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr uint32_t idesc = idesc_e4m3(P8_BM, P8_BN);
            const bool issues = elect_one();
            Ring<P8_STAGES> r;
            uint32_t local = 0;
            bool ok = true;
            for (long long t = first; t < tiles && ok; t += step, ++local) {
                const uint32_t a = local & 1;
                if (local >= 2 && !warp_wait(&tm_empty[a], ((local >> 1) & 1) ^ 1, limit)) break;
                tc_fence_after();
                const uint32_t acc = tmem + a * P8_BN;
                for (int kb = 0; kb < KB; ++kb, r.next()) {
                    if (!warp_wait(&full[r.s], r.round, limit)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_addr(smem + r.s * P8_STAGE);
                    if (issues) {
                        mma_block<2>(acc, sa, sa + P8_HALF, idesc, kb);
                        commit_pair(&empty[r.s]);
                    }
                }
                if (ok && issues) commit_pair(&tm_full[a]);
            }
            if (issues) commit_pair(drained);
            __syncwarp();
        }
        // the MMAs complete, and their arrivals are here, before a CTA can leave, whether or not its epilogue waited
        for (long long t = first; t < tiles && !warp_wait(drained, 0, WAIT_LIMIT_DEFAULT); t += step) {
        }
    } else {
        const int q = warp & 3;            // TMEM lane quarter this warp may access
        const int part = (warp - 2) >> 2;  // 64 columns of the tile
        uint8_t *buf = smem + P8_OUT + (warp - 2) * P8_TILE;
        uint32_t local = 0;
        bool gave_up = false;
        for (long long t = first; t < tiles; t += step, ++local) {
            const uint32_t a = local & 1;
            const int y = (int)(t / tiles_n) * P8_BM + (int)rank * 128 + q * 32, n0 = (int)(t % tiles_n) * P8_BN + part * 64;
            RowScale sx(y + lane < M ? __ldg(xs + y + lane) : 0.0f);
            // 16 columns' scales, the first ones while the MMAs run; columns past N, a multiple of 16,
            // take others' and are not stored
            float4 w[4];
            auto read_scales = [&](int col) {
                const float4 *p = reinterpret_cast<const float4 *>(ws + min(col, N - 16));
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = __ldg(p + j);
            };
            read_scales(n0);
            // a wait that gave up leaves NaN in this tile and in those after it (added to a residual, too)
            gave_up = gave_up || !warp_poll(&tm_full[a], (local >> 1) & 1, limit);
            if (gave_up) sx.s = __uint_as_float(NAN_BITS);
            tc_fence_after();
            const uint32_t t_row = tmem + a * P8_BN + part * 64 + ((uint32_t)(q * 32) << 16);
            // the tile's rows of 64 bytes: 16-byte piece u of row r at u ^ (r / 2) % 4 (64-byte swizzle)
            uint8_t *out_row = buf + lane * 64;
            const int sw = (lane >> 1) & 3;
            auto buffer_free = [&]() {  // the last store has read it
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
            };
            auto store_tile = [&](int col, bool inside) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0 && inside) tile_out<EPI == EPI_RESID_ADD>(&tmO, buf, col, y);
                if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            };
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int col = n0 + c * 16;
                uint32_t x[16];
                tmem_ld16(t_row + c * 16, x);
                if (c == 3) {  // the accumulator has been read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0 && !gave_up) arrive_at(in_cta(&tm_empty[a], 0));
                }
                float2 v[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 s2 = make_float2(sx.s, sx.s);
                    v[2 * j] = mul2(mul2(make_float2(__uint_as_float(x[4 * j]), __uint_as_float(x[4 * j + 1])), s2),
                                    make_float2(w[j].x, w[j].y));
                    v[2 * j + 1] = mul2(mul2(make_float2(__uint_as_float(x[4 * j + 2]), __uint_as_float(x[4 * j + 3])), s2),
                                        make_float2(w[j].z, w[j].w));
                }
                if (sx.f != 1.0f)
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = mul2(v[j], make_float2(sx.f, sx.f));
                if (c < 3) read_scales(col + 16);
                if (EPI == EPI_SWIGLU) {  // 16 columns are one piece of the tile's rows
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = pack_bf16x2(swiglu(v[2 * j].x, v[2 * j].y), swiglu(v[2 * j + 1].x, v[2 * j + 1].y));
                    if (c == 0) buffer_free();
                    *reinterpret_cast<uint4 *>(out_row + ((c ^ sw) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                    if (c == 3) store_tile(n0 / 2, y < M && n0 < N);
                } else {  // or the whole tile
                    buffer_free();
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<float4 *>(out_row + ((j ^ sw) << 4)) =
                            make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
                    store_tile(col, y < M && col < N);
                }
            }
        }
        if (lane == 0) tma_store_wait_all();  // the tiles are in global memory
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA's shared or tensor memory is in use
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// 2-D map of the output as tiles of 32 rows of 64 bytes: fp32 [rows, cols], or bf16 for SwiGLU.
bool make_map_out(CUtensorMap *map, void *base, int rows, int cols, bool half) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)cols * (half ? 2 : 4)};
    const cuuint32_t box[2] = {half ? 32u : 16u, 32};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, half ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, base, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int EPI>
cudaError_t run_pair(const Launch &lc, const uint8_t *xq, const float *xs, int M, int K, const uint8_t *wq, const float *ws,
                     int N, void *out) {
    CUtensorMap ma, mb, mo;
    if (!make_map_q8(&ma, xq, M, K, 128) || !make_map_q8(&mb, wq, N, K, 128) ||
        !make_map_out(&mo, out, M, EPI == EPI_SWIGLU ? N / 2 : N, EPI == EPI_SWIGLU))
        return cudaErrorInvalidValue;
    static SharedLimit limit;
    const cudaError_t e = limit.raise(k_gemm_q8_pair<EPI>, P8_SMEM);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)((M + P8_BM - 1) / P8_BM) * ((N + P8_BN - 1) / P8_BN);
    const int pairs = (int)(tiles < lc.num_sms / 2 ? tiles : lc.num_sms / 2);
    return launch(lc, k_gemm_q8_pair<EPI>, dim3(2 * pairs), dim3(P8_THREADS), P8_SMEM, ma, mb, mo, xs, ws, M, N, K,
                  lc.wait_limit);
}

template <int BN, int EPI, bool SPLIT>
cudaError_t run_q8(const Launch &lc, const uint8_t *xq, const float *xs, int M, int K, const uint8_t *wq, const float *ws,
                   int N, void *out, int S) {
    CUtensorMap ma, mb;
    if (!make_map_q8(&ma, xq, M, K, (int)q8_box_rows(M)) || !make_map_q8(&mb, wq, N, K, BN)) return cudaErrorInvalidValue;
    static SharedLimit limit;
    const cudaError_t e = limit.raise(k_gemm_q8<BN, EPI, SPLIT>, G8<BN>::SMEM);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)((M + G8_BM - 1) / G8_BM) * ((N + BN - 1) / BN);
    if (SPLIT)
        return launch_cluster(lc, k_gemm_q8<BN, EPI, SPLIT>, dim3((unsigned)(tiles * S)), dim3(G8_THREADS), G8<BN>::SMEM,
                              dim3(S, 1, 1), ma, mb, xs, ws, M, N, K, out, S, lc.wait_limit);
    const int grid = (int)(tiles < lc.num_sms ? tiles : lc.num_sms);
    return launch(lc, k_gemm_q8<BN, EPI, SPLIT>, dim3(grid), dim3(G8_THREADS), G8<BN>::SMEM, ma, mb, xs, ws, M, N, K, out, 1,
                  lc.wait_limit);
}
template <int BN, int EPI>
cudaError_t run_single(const Launch &lc, const uint8_t *xq, const float *xs, int M, int K, const uint8_t *wq, const float *ws,
                       int N, void *out, int S) {
    return S > 1 ? run_q8<BN, EPI, true>(lc, xq, xs, M, K, wq, ws, N, out, S)
                 : run_q8<BN, EPI, false>(lc, xq, xs, M, K, wq, ws, N, out, 1);
}

// The form, tile and split of K whose estimate is lowest.  In clocks past a launch's own, fitted to 1199
// timed launches of 1 to 4,096 rows, K 512 to 24,576, N 272 to 8,192 (10% rms; what it picks is 0.8%
// slower than the best of them on average, 23% at worst, where residuals of 200 rows bound it; not fitted again since
// SwiGLU and the scales were changed):
//   a k-block of a single CTA: 300 for its waits and issue, or 1.37 a row of its operands;
//   a single CTA's tile: 160 + 10.3 a column + 0.29 an output, half hidden by the next tile's MMAs;
//   joining a split tile: 2,000;  a k-block of a pair 555, its first and last tile 7,450.
// Both sides, in us: 33 x 1024 x 2048 with the residual 5.1 whole, 4.7 in 4 shares of K; x 8192 12.0 and
// 6.0 (8 shares); x 24576 30.9 and 9.2; 33 x 1024 x 1024 3.9 and 4.3.  600 x 6144 x 1024 17.9 in single
// CTAs, 9.8 in pairs; 600 x 2048 x 2048 8.2 and 10.4.
Q8Plan choose_q8(int num_sms, int M, int K, int N) {
    const long long kb = (K + G8_BK - 1) / G8_BK, rows = q8_box_rows(M), live = M < 128 ? M : 128;
    auto up = [](long long a, long long b) { return (a + b - 1) / b; };
    long long best = up(up(M, P8_BM) * up(N, P8_BN), num_sms / 2) * kb * 555 + 7450;
    Q8Plan plan;
    for (int b = 32; b <= 128; b *= 2)
        for (int s = 1; s <= MAX_SPLIT && s <= kb; s *= 2) {
            const long long tiles = up(M, G8_BM) * up(N, b);
            // CTAs at once: the GPCs of 152 SMs hold 36 clusters of 4 and 15 of 8
            const long long at_once = s == 8 ? num_sms * 15 / 19 : s == 4 ? num_sms * 18 / 19 : num_sms;
            if (s > 1 && tiles * s > at_once) break;
            const long long block = (rows + b) * 137 / 100, loop = up(kb, s) * (block > 300 ? block : 300);
            const long long tile = 160 + b * 103 / 10 + live * b * 29 / 100, n = up(tiles * s, at_once);
            const long long clocks = n * loop + (n + 1) * tile / 2 + (s > 1 ? 2000 : 0);
            if (clocks < best) {
                best = clocks;
                plan.tile_cols = b;
                plan.k_shares = s;
            }
        }
    return plan;
}

template <int EPI>
cudaError_t run_plan(const Launch &lc, const uint8_t *xq, const float *xs, int M, int K, const uint8_t *wq, const float *ws,
                     int N, void *out) {
    const Q8Plan plan = choose_q8(lc.num_sms, M, K, N);
    switch (plan.tile_cols) {
        case 256: return run_pair<EPI>(lc, xq, xs, M, K, wq, ws, N, out);
        case 128: return run_single<128, EPI>(lc, xq, xs, M, K, wq, ws, N, out, plan.k_shares);
        case 64: return run_single<64, EPI>(lc, xq, xs, M, K, wq, ws, N, out, plan.k_shares);
        default: return run_single<32, EPI>(lc, xq, xs, M, K, wq, ws, N, out, plan.k_shares);
    }
}

}  // namespace

Q8Plan plan_gemm_q8(int num_sms, int M, int K, int N) { return choose_q8(num_sms, M, K, N); }

cudaError_t launch_gemm_q8(const Launch &lc, const uint8_t *xq, const float *xs, int M, int K, const uint8_t *wq,
                           const float *ws, int N, int epi, void *out) {
    switch (epi) {
        case EPI_F32: return run_plan<EPI_F32>(lc, xq, xs, M, K, wq, ws, N, out);
        case EPI_RESID_ADD: return run_plan<EPI_RESID_ADD>(lc, xq, xs, M, K, wq, ws, N, out);
        case EPI_SWIGLU: return run_plan<EPI_SWIGLU>(lc, xq, xs, M, K, wq, ws, N, out);
    }
    return cudaErrorInvalidValue;
}

}  // namespace q3
