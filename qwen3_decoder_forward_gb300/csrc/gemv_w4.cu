// Decode projection on 4-bit weights: out[M,N] = x[M,K] . W[N,K]^T with W = s (code - z) per group of
// G columns, for up to 32 rows of x a launch.  What it cannot do without is streaming the codes, and it does not
// reach that.  A box of 8,192 codes and up to 8 rows of x takes some 715 instructions, half of them to make bf16
// fragments of codes: with 16 warps an SM their issue takes 58% of the slots (2 rows of the head, IPC 2.3).  From 9 rows
// on, with 8 warps an SM and 96 to 144 of 152 SMs in use, a warp waits on its own chain of conversion and mma.sync (13
// rows: IPC 1.5, no pipe above 30%).  In us, with the floor: one row of a 151,936 x 1024 head 19.2 (12.1), one of
// 8,192 x 10,240 13.2 (6.5), 13 rows of it 21.8 (6.7), 32 of 16,384 x 4,096 28 (5.5), one of 4096 x 1024 a launch's 3.0.
//
// Sum over a row of W:  sum_groups s_g sum_{k in g} (code_k - z_g) x_k.  code - z is a small integer,
// exact in bf16, so the inner sums run on the tensor cores (mma.sync m16n8k16, weight rows as the
// M side, rows of x as the N side) and a group's sum is multiplied by its scale in fp32.
//   A 32-bit word holds 8 codes of one row: (w >> 4i) & 0x000f000f | 0x43004300 is the bf16 pair
// (128 + code_i, 128 + code_{i+4}), and one exact packed subtraction of 128 + z leaves the A
// fragment (integers made floats by setting the exponent above their bits, as published for weights of few bits by
// Kim, Henry, Fahim and Awadalla, "Who Says Elephants Can't Run", 2022).  x is staged once per CTA as bf16 (exact from
// e4m3) with every 8 columns in the matching order (0,4,1,5,2,6,3,7), so the B fragments of two steps are one
// 16-byte read.
//   A 32-row tile of W moves in boxes of 256 columns (128 bytes a row) by TMA into a ring of
// the warp's own, swizzled so that the 32 lanes' 4-byte reads (8 rows x 4 words of one 16-byte piece)
// touch 32 banks.
//   The warps of a CTA are row tiles by WK shares of the columns; a cluster of CTAs may share
// the columns further, each staging its own columns of x only.  Shares meet in shared memory
// (distributed, across a cluster) in a fixed order: no atomics, the same bits on every run.

#include <cuda.h>
#include <cuda_fp8.h>

#include <cmath>

#include "kernels.h"
#include "tc.cuh"

namespace q3 {

namespace {

constexpr int W4_BK = 256;            // columns of a box: 128 bytes of codes
constexpr int W4_ROWS = 32;           // rows of W of a box
constexpr int W4_BOX = W4_ROWS * 128;  // bytes of a box
constexpr int W4_ST = 2;              // boxes in flight per warp
constexpr int W4_SMEM_MAX = 227 * 1024;

struct W4Args {
    const void *x;
    const float *xs;
    const bf16 *scales;
    const uint8_t *zeros;
    void *out;
    int M, K, N, epi;
    int NW;        // warps of a CTA
    int WK;        // column shares within a CTA (NW / WK row tiles of 32)
    int S;         // CTAs of a cluster sharing the columns
    int kslice;    // columns of a CTA of the cluster, a multiple of 256
    int xstride;   // bytes of a staged row of x, 64 modulo 128
    long long limit;  // of a wait, in clocks
};

// MT: 8-row tiles of x.
template <bool ZEROS, int G, int MT>
struct W4 {
    static constexpr int MAX_WARPS = MT <= 2 ? 16 : 8;  // by registers
    static constexpr int NG = W4_BK / G;                // groups of a box
    // Scales and zero points of a box, 4-byte words of each row: its NG values may start and end
    // inside a word.
    static constexpr int SW = NG / 2 + 1, ZW = ZEROS ? (NG + 2) / 4 + 1 : 0;
    static constexpr int SC = (SW + ZW) * W4_ROWS;
    // Partial sums of a tile [warp][row of x][row of W]: 36 floats apart, so that a fragment's stores
    // touch 32 banks, and neighbouring outputs are neighbours for whoever joins them.
    static constexpr int RP = W4_ROWS + 4, SHARE = MT * 8 * RP;
    // Shared memory: the warps' boxes; barriers and row scales; then each warp's scales and sums.
    static constexpr int PER_WARP = W4_ST * W4_BOX + W4_ST * SC * 4 + SHARE * 4;
    static constexpr int FIXED = 512 + 1024;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The same place of shared memory in CTA `rank` of the cluster (generic addresses).
__device__ __forceinline__ const float *in_cta(const float *p, uint32_t rank) {
    uint64_t q;
    asm("mapa.u64 %0, %1, %2;" : "=l"(q) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
    return reinterpret_cast<const float *>(q);
}

__device__ __forceinline__ void add_to(float &v, float y) { v += y; }
__device__ __forceinline__ void add_to(float2 &v, float2 y) {
    v.x += y.x;
    v.y += y.y;
}

// c = a b
__device__ __forceinline__ void mma_bf16_first(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// c += a b
__device__ __forceinline__ void mma_bf16(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes i and i + 4 of w minus the zero point: zc is the bf16 pair (128 + z, 128 + z).  One lop3 takes
// the nibbles and sets the exponents (written as two operators it became two instructions).
template <int I>
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, uint32_t zc) {
    uint32_t t;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(t) : "r"(w >> (4 * I)), "r"(0x000f000fu), "r"(0x43004300u));
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&t),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&zc));
    return *reinterpret_cast<const uint32_t *>(&d);
}

// Words of a row's values from element `at` on of an array of `values` elements of BYTES,
// asynchronously, from the word that holds it; bytes past the array's end become zero.
template <int BYTES, int WORDS>
__device__ __forceinline__ void copy_words(uint32_t *to, const void *array, long long at, long long values) {
    const long long byte = (at * BYTES) & ~3ll;
    const uint8_t *from = static_cast<const uint8_t *>(array) + byte;
    const uint32_t dst = smem_addr(to);
    if (byte + WORDS * 4 <= values * BYTES) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst + 4 * i), "l"(from + 4 * i) : "memory");
    } else {  // the array's last row, or a row past it
        const int left = (int)max(0ll, values * BYTES - byte);
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            const int n = min(4, max(0, left - 4 * i));
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + 4 * i),
                         "l"(n > 0 ? from + 4 * i : static_cast<const uint8_t *>(array)), "r"(n)
                         : "memory");
        }
    }
}

// Eight columns of x from element i on, as read.
template <bool XQ>
__device__ __forceinline__ uint4 read_x8(const void *x, size_t i) {
    if (!XQ) return __ldg(reinterpret_cast<const uint4 *>(static_cast<const bf16 *>(x) + i));
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(x) + i));
    return make_uint4(u.x, u.y, 0, 0);
}

// The same as four bf16 pairs (0,4), (1,5), (2,6), (3,7).
template <bool XQ>
__device__ __forceinline__ uint4 pairs_x8(uint4 u) {
    if (XQ) {
        const uint32_t w[2] = {u.x, u.y};
        uint32_t p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j / 2] >> (16 * (j & 1))), __NV_E4M3);
            const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            p[j] = pack_bf16x2(t.x, t.y);  // exact: 4 significant bits
        }
        u = make_uint4(p[0], p[1], p[2], p[3]);
    }
    return make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632), __byte_perm(u.y, u.w, 0x5410),
                      __byte_perm(u.y, u.w, 0x7632));
}

template <bool XQ, bool ZEROS, int G, int MT>
__global__ void __launch_bounds__(W4<ZEROS, G, MT>::MAX_WARPS * 32, 1)
    k_gemv_w4(const __grid_constant__ CUtensorMap tm, const W4Args a) {
    using T = W4<ZEROS, G, MT>;
    constexpr int RM = 2;  // 16-row tiles of a box
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *head = smem + a.NW * W4_ST * W4_BOX;                  // after the boxes
    uint64_t *bars = reinterpret_cast<uint64_t *>(head);           // [warps][ST]
    uint32_t *scs = reinterpret_cast<uint32_t *>(head + 512);      // [warps][ST][SC]
    float *red = reinterpret_cast<float *>(scs + a.NW * W4_ST * T::SC);
    uint8_t *xsm = reinterpret_cast<uint8_t *>(red + a.NW * T::SHARE);
    float *xsc = reinterpret_cast<float *>(head + 384);  // row scales of x

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const int rank = a.S > 1 ? (int)cluster_rank() : 0;
    const int NT = a.NW * 32, WN = a.NW / a.WK, wn = warp / a.WK, wk = warp % a.WK;
    const int tile_rows = WN * W4_ROWS;
    const int tiles = (a.N + tile_rows - 1) / tile_rows;
    const int first = blockIdx.x / a.S, step = gridDim.x / a.S;
    const int k_lo = rank * a.kslice, k_hi = min(a.K, k_lo + a.kslice);
    // this warp's boxes of a tile: columns k_lo + 256 (wk + j WK)
    const int boxes = k_hi > k_lo ? (k_hi - k_lo + W4_BK - 1) / W4_BK : 0;
    const int mine = boxes > wk ? (boxes - wk + a.WK - 1) / a.WK : 0;
    const int my_tiles = (tiles - first + step - 1) / step;  // at least one: the grid has no more clusters than tiles
    const int units = mine * my_tiles;
    const int ng = a.K / G;

    uint8_t *ring = smem + warp * W4_ST * W4_BOX;
    uint64_t *full = bars + warp * W4_ST;
    uint32_t *sc = scs + warp * W4_ST * T::SC;

    if (lane == 0)
        for (int s = 0; s < W4_ST; ++s) mbar_init(&full[s], 1 + 32);  // the codes; each lane's row of scales
    __syncwarp();

    // The next box to fetch: its row of W, place among the tile's boxes, and the index of its
    // first scale in this lane's row.
    int f_row = first * tile_rows + wn * W4_ROWS, f_j = 0;
    const int g_first = (k_lo + wk * W4_BK) / G, g_step = a.WK * T::NG;
    const long long values = (long long)a.N * ng;  // scales, zero points
    long long f_at = (long long)(f_row + lane) * ng + g_first;
    auto fetch = [&](int s) {
        if (lane == 0) {
            mbar_expect_tx(&full[s], W4_BOX);  // rows and columns past the end are zero-filled
            tma_load_2d(ring + s * W4_BOX, &tm, (k_lo + (wk + f_j * a.WK) * W4_BK) / 2, f_row, &full[s]);
        }
        uint32_t *to = sc + s * T::SC;
        copy_words<2, T::SW>(to + lane * T::SW, a.scales, f_at, values);
        if (ZEROS) copy_words<1, T::ZW>(to + T::SW * W4_ROWS + lane * T::ZW, a.zeros, f_at, values);
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&full[s])) : "memory");
        f_at += g_step;
        if (++f_j == mine) {
            f_j = 0;
            f_row += step * tile_rows;
            f_at = (long long)(f_row + lane) * ng + g_first;
        }
    };
    pdl_wait();  // the weights, too, may be the previous kernel's output
    pdl_trigger();
    for (int u = 0; u < min(units, W4_ST); ++u) fetch(u);

    // x, this CTA's columns
    if (XQ && (int)threadIdx.x < a.M) xsc[threadIdx.x] = a.xs[threadIdx.x];
    {
        // in pieces of 256 columns, 8 a lane, dealt to the warps in turn
        constexpr int BATCH = 8;  // loads in flight of a thread
        const int per_row = max(0, k_hi - k_lo) / 8, pieces = (per_row + 31) / 32;
        int m = 0, c = warp;
        auto settle = [&]() {
            while (c >= pieces && m < a.M) {
                c -= pieces;
                ++m;
            }
        };
        settle();
        while (m < a.M) {
            uint4 raw[BATCH];
            uint32_t to[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int v = c * 32 + lane;
                to[b] = 0xffffffffu;
                if (m < a.M && v < per_row) {
                    raw[b] = read_x8<XQ>(a.x, (size_t)m * a.K + k_lo + v * 8);
                    to[b] = (uint32_t)(m * a.xstride + v * 16);
                }
                c += a.NW;
                settle();
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b)
                if (to[b] != 0xffffffffu) *reinterpret_cast<uint4 *>(xsm + to[b]) = pairs_x8<XQ>(raw[b]);
        }
    }
    __syncthreads();

    // rows of x past M read the last one's: a column of the product depends on its own row alone
    uint32_t xrow[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) xrow[t] = smem_addr(xsm) + (uint32_t)(min(t * 8 + g, a.M - 1) * a.xstride + t4 * 16);

    // 16-byte piece of block b (of a quarter of the box) in this lane's rows, under the swizzle
    uint32_t piece[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) piece[b] = (uint32_t)((b ^ (g & 3)) << 4);

    bool ok = true;
    int u = 0;
    for (int i = 0; i < my_tiles; ++i) {
        float acc[RM][MT][4];
#pragma unroll
        for (int r = 0; r < RM; ++r)
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[r][t][e] = 0.0f;
        // Byte of the first value in each row's words of scales and zero points (WK NG boxes' values
        // on: even, so the scales' phase holds for the tile)
        uint32_t soff[RM][2], zph[RM][2];
#pragma unroll
        for (int r = 0; r < RM; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = r * 16 + h * 8 + g;
                const uint32_t at = (uint32_t)((first + i * step) * tile_rows + wn * W4_ROWS + row) * (uint32_t)ng +
                                    (uint32_t)((k_lo + wk * W4_BK) / G);
                soff[r][h] = row * T::SW * 4 + (at & 1) * 2;
                zph[r][h] = at;
            }
        for (int j = 0; j < mine && ok; ++j, ++u) {
            const int s = u % W4_ST;
            const uint32_t phase = (u / W4_ST) & 1;
            if (!warp_poll(&full[s], phase, a.limit)) {
                ok = false;
                break;
            }
            const int kx = (wk + j * a.WK) * W4_BK;  // within the staged columns
            const uint32_t box = smem_addr(ring + s * W4_BOX) + g * 128 + t4 * 4;
            const uint32_t scw = smem_addr(sc + s * T::SC), zpw = scw + T::SW * W4_ROWS * 4;
            const int groups = min(T::NG, (k_hi - k_lo - kx) / G);
#pragma unroll 1
            for (int gi = 0; gi < groups; ++gi) {
                float part[RM][MT][4];
                float scale[RM][2];
                uint32_t zc[RM][2];
#pragma unroll
                for (int r = 0; r < RM; ++r)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint16_t v;
                        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(scw + soff[r][h] + gi * 2));
                        scale[r][h] = __uint_as_float((uint32_t)v << 16);
                        uint32_t z = 8;
                        if (ZEROS) {
                            const uint32_t ph = (zph[r][h] + j * a.WK * T::NG) & 3;
                            asm volatile("ld.shared.u8 %0, [%1];"
                                         : "=r"(z)
                                         : "r"(zpw + (r * 16 + h * 8 + g) * T::ZW * 4 + ph + gi));
                            z &= 15;
                        }
                        zc[r][h] = z * 0x00010001u + 0x43004300u;
                    }
                const uint32_t quarter = G == 128 ? box + ((gi ^ (g >> 2)) << 6) : 0;
#pragma unroll
                for (int b = 0; b < G / 32; ++b) {
                    const int blk = gi * (G / 32) + b;
                    const uint32_t at = G == 128 ? quarter + piece[b] : box + ((blk ^ g) << 4);
                    uint32_t fr[RM][2][4];
#pragma unroll
                    for (int r = 0; r < RM; ++r) {
                        uint32_t w[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            asm volatile("ld.shared.u32 %0, [%1];"
                                         : "=r"(w[h])
                                         : "r"(at + (r * 16 + h * 8) * 128));
#pragma unroll
                        for (int h = 0; h < 2; ++h) {  // registers h (first pair) and h + 2 (second) of each step
                            fr[r][0][h] = w4_pair<0>(w[h], zc[r][h]);
                            fr[r][0][h + 2] = w4_pair<1>(w[h], zc[r][h]);
                            fr[r][1][h] = w4_pair<2>(w[h], zc[r][h]);
                            fr[r][1][h + 2] = w4_pair<3>(w[h], zc[r][h]);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        uint32_t x0, x1, x2, x3;
                        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(x0), "=r"(x1), "=r"(x2), "=r"(x3)
                                     : "r"(xrow[t] + kx * 2 + blk * 64));
#pragma unroll
                        for (int r = 0; r < RM; ++r) {
                            if (b == 0)
                                mma_bf16_first(part[r][t], fr[r][0], x0, x1);
                            else
                                mma_bf16(part[r][t], fr[r][0], x0, x1);
                            mma_bf16(part[r][t], fr[r][1], x2, x3);
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < RM; ++r)
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[r][t][e] = fmaf(scale[r][e >> 1], part[r][t][e], acc[r][t][e]);
            }
            __syncwarp();  // every lane has read the box and the scales of this unit
            if (u + W4_ST < units) fetch(s);
        }
        if (!ok) {  // a wait gave up: the outputs say so
#pragma unroll
            for (int r = 0; r < RM; ++r)
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[r][t][e] = __uint_as_float(0x7fffffffu);
        }
        if (a.WK == 1 && a.S == 1) {
            // the warp has its rows' whole sums: straight to the output, no join (head, 2 rows: 22.7 ->
            // 20.9 us; 16 rows of 100,000 x 1,024: 28.8 -> 19.9; eight lanes of a fragment are eight neighbouring outputs)
            const int n0 = (first + i * step) * tile_rows + wn * W4_ROWS + g;
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int m = t * 8 + t4 * 2 + e;
                    const float sx = XQ && m < a.M ? xsc[m] : 1.0f;
                    float v[RM * 2];
                    size_t at[RM * 2];
#pragma unroll
                    for (int r = 0; r < RM * 2; ++r) {
                        v[r] = acc[r / 2][t][(r & 1) * 2 + e] * sx;
                        at[r] = (size_t)m * a.N + n0 + r * 8;
                    }
                    if (a.epi == EPI_SWIGLU) {  // lanes of odd rows hold up, their neighbours gate
#pragma unroll
                        for (int r = 0; r < RM * 2; ++r) {
                            const float up = __shfl_xor_sync(0xffffffffu, v[r], 4);
                            if (!(g & 1) && m < a.M && n0 + r * 8 < a.N)
                                static_cast<bf16 *>(a.out)[(size_t)m * (a.N / 2) + (n0 + r * 8) / 2] = __float2bfloat16(swiglu(v[r], up));
                        }
                    } else {
                        float *o = static_cast<float *>(a.out);
                        if (a.epi == EPI_RESID_ADD) {
#pragma unroll
                            for (int r = 0; r < RM * 2; ++r)
                                if (m < a.M && n0 + r * 8 < a.N) v[r] += o[at[r]];
                        }
#pragma unroll
                        for (int r = 0; r < RM * 2; ++r)
                            if (m < a.M && n0 + r * 8 < a.N) o[at[r]] = v[r];
                    }
                }
            continue;
        }
        // each CTA of the cluster finishes its share of the tile's rows; the residual that a thread
        // adds to first is read while the shares meet
        const int rows = tile_rows / a.S, n0 = (first + i * step) * tile_rows + rank * rows;
        const int per = a.epi == EPI_SWIGLU ? 2 : 1, outs = rows / per;
        float held = 0.0f;
        if (a.epi == EPI_RESID_ADD && (int)threadIdx.x < outs * a.M) {
            const int m = threadIdx.x / outs, n = n0 + (threadIdx.x - m * outs);
            if (n < a.N) held = static_cast<const float *>(a.out)[(size_t)m * a.N + n];
        }
        // shares of the tile: [warp][row][x row]
        __syncwarp();
        if (i > 0) {  // the last tile's shares have been read
            if (a.S > 1)
                cluster_wait();
            else
                __syncthreads();
        }
#pragma unroll
        for (int r = 0; r < RM; ++r)
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                float *p = red + warp * T::SHARE + (t * 8 + t4 * 2) * T::RP + r * 16 + g;
                p[0] = acc[r][t][0];
                p[T::RP] = acc[r][t][1];
                p[8] = acc[r][t][2];
                p[T::RP + 8] = acc[r][t][3];
            }
        if (a.S > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        auto total = [&](int r, int m, auto zero) {  // rows r (and r + 1) of the tile
            using V = decltype(zero);
            const float *p = red + r / W4_ROWS * a.WK * T::SHARE + m * T::RP + r % W4_ROWS;
            V v = zero;
            for (int c = 0; c < a.S; ++c) {
                const float *q = a.S > 1 ? in_cta(p, c) : p;
                if (a.WK == 1) {
                    add_to(v, *reinterpret_cast<const V *>(q));
                } else {
#pragma unroll 4
                    for (int w = 0; w < a.WK; w += 2) {
                        const V y0 = *reinterpret_cast<const V *>(q + w * T::SHARE);
                        const V y1 = *reinterpret_cast<const V *>(q + (w + 1) * T::SHARE);
                        add_to(v, y0);
                        add_to(v, y1);
                    }
                }
            }
            return v;
        };
        for (int e = threadIdx.x; e < outs * a.M; e += NT) {
            const int m = e / outs, r = (e - m * outs) * per, n = n0 + r;
            if (n >= a.N) continue;
            const float sx = XQ ? xsc[m] : 1.0f;
            if (a.epi == EPI_SWIGLU) {
                const float2 v = total(rank * rows + r, m, make_float2(0.0f, 0.0f));
                static_cast<bf16 *>(a.out)[(size_t)m * (a.N / 2) + n / 2] = __float2bfloat16(swiglu(v.x * sx, v.y * sx));
            } else {
                const float v = total(rank * rows + r, m, 0.0f) * sx;
                float *o = static_cast<float *>(a.out) + (size_t)m * a.N + n;
                *o = a.epi != EPI_RESID_ADD ? v : v + (e == (int)threadIdx.x ? held : *o);
            }
        }
        __syncwarp();
        if (a.S > 1) cluster_arrive();  // this tile's shares have been read
    }
    if (a.S > 1) {
        cluster_wait();  // no CTA leaves while another reads its shares
    }
    if (!ok)  // copies in flight land before the CTA leaves
        for (int v = u; v < min(units, u + W4_ST); ++v) mbar_wait_bounded(&full[v % W4_ST], (v / W4_ST) & 1, nullptr);
}

int x_stride(int kslice) { return kslice * 2 + 64; }
int x_bytes(int m, int kslice) { return m * x_stride(kslice); }  // shared memory of m rows of x

// The cheapest cut by an estimate: x staged once per CTA, then rounds of tiles, each bound by the
// warps' issue rate or by latency, and closed by a join (none where a warp has its rows' whole sums).
// The constants were fitted to all cuts of 23 sizes (1 to 32 rows, K 256 to 16,384, N 500 to
// 151,936): its choice was 1% slower than the best cut on average and 7% at worst, before launches overlapped and
// x was staged by whole warps; not fitted again since.  It is low where x's staging counts: 32 x 6144 x 1024 4.7 us
// against 7.6, 32 x 16,384 x 4,096 21.4 against 28.  8 warps sharing
// a 32-row tile's columns, without clusters, are up to 2.2 times slower (32 rows, 100,000 x 1,024:
// 64 against 29 us; 1 row, 500 x 16,384: 13.3 against 6.9).
W4Plan plan_w4(int num_sms, int M, int K, int N, int mt, int max_warps, int fixed, int per_warp) {
    const int boxes = (K + W4_BK - 1) / W4_BK;
    W4Plan best;
    for (int NW = 8; NW <= max_warps; NW += 4)
        for (int S = 1; S <= 8; S *= 2) {
            if (S > 1 && S > boxes) break;
            W4Plan p;
            p.NW = NW;
            p.S = S;
            const int slice = (boxes + S - 1) / S;
            p.kslice = slice * W4_BK;
            const int smem = fixed + NW * per_warp + x_bytes(M, p.kslice);
            if (smem > W4_SMEM_MAX) continue;
            // by shared memory; 128 registers a thread (256 with 4 row tiles of x)
            const int per_sm = NW == 8 && mt <= 2 && 2 * (smem + 1024) <= 228 * 1024 ? 2 : 1;
            // clusters that run at once: the GPCs hold 36 of 4 and 15 of 8 at one CTA an SM
            const int slots = num_sms * per_sm * (S == 8 ? 79 : S == 4 ? 95 : 100) / 100 / S;
            for (p.WK = 1; p.WK <= NW && p.WK <= slice; p.WK *= 2) {
                if (NW % p.WK) break;
                p.tile_rows = W4_ROWS * (NW / p.WK);
                const int tiles = (N + p.tile_rows - 1) / p.tile_rows;
                p.clusters = tiles < slots ? tiles : slots;
                p.rounds = (tiles + p.clusters - 1) / p.clusters;
                const int resident = (p.clusters * S + num_sms - 1) / num_sms;  // CTAs of the busiest SM
                const int warps = resident * NW;
                const int mine = (slice + p.WK - 1) / p.WK;  // boxes of a warp and tile
                const float box_ns = (744 + 45 * mt) / 1.9f / (warps >= 12 ? 2.4f : 2.28f);
                const float tile_ns = fmaxf((float)mine * warps * box_ns, 700.0f + 300.0f * mine);
                const float join_ns = S > 1 ? 2550.0f : p.WK > 1 ? 255.0f + 49.0f * mt : 50.0f;
                p.ns = 1360.0f + 17.0f * warps + (float)x_bytes(M, p.kslice) * resident / 70.0f +
                       p.rounds * (tile_ns + join_ns + 20.0f * p.WK * S);
                if (!best.NW || p.ns < best.ns) best = p;
            }
        }
    return best;
}

// 2-D map of the codes [N][K / 2] as boxes of 128 bytes x 32 rows, 128-byte swizzle.
bool make_map_w4(CUtensorMap *map, const uint8_t *codes, int N, int K) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)N};
    const cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
    const cuuint32_t box[2] = {128, W4_ROWS};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool ZEROS, int G, int MT>
W4Plan plan_for(int num_sms, int M, int K, int N) {
    using T = W4<ZEROS, G, MT>;
    return plan_w4(num_sms, M, K, N, MT, T::MAX_WARPS, T::FIXED, T::PER_WARP);
}
template <bool ZEROS, int G>
W4Plan plan_rows(int num_sms, int M, int K, int N) {
    return M <= 8 ? plan_for<ZEROS, G, 1>(num_sms, M, K, N)
                  : M <= 16 ? plan_for<ZEROS, G, 2>(num_sms, M, K, N) : plan_for<ZEROS, G, 4>(num_sms, M, K, N);
}

// Rows of x a launch: 32, fewer where a cluster of 8 CTAs cannot hold 32 of this length.
int pass_rows(int K) {
    const int slice = ((K + W4_BK - 1) / W4_BK + 7) / 8 * W4_BK;
    return x_bytes(32, slice) <= 96 * 1024 ? 32 : x_bytes(16, slice) <= 96 * 1024 ? 16 : 8;
}

template <bool XQ, bool ZEROS, int G, int MT>
cudaError_t run_w4(const Launch &lc, W4Args a, const uint8_t *codes) {
    using T = W4<ZEROS, G, MT>;
    const W4Plan p = plan_for<ZEROS, G, MT>(lc.num_sms, a.M, a.K, a.N);
    if (!p.NW) return cudaErrorInvalidValue;
    a.NW = p.NW;
    a.S = p.S;
    a.WK = p.WK;
    a.kslice = p.kslice;
    a.xstride = x_stride(p.kslice);
    const int smem = T::FIXED + p.NW * T::PER_WARP + x_bytes(a.M, p.kslice);
    CUtensorMap tm;
    if (!make_map_w4(&tm, codes, a.N, a.K)) return cudaErrorInvalidValue;
    auto kern = k_gemv_w4<XQ, ZEROS, G, MT>;
    static SharedLimit limit;
    const cudaError_t e = limit.raise(kern, W4_SMEM_MAX);
    if (e != cudaSuccess) return e;
    const dim3 grid(p.clusters * p.S), block(p.NW * 32);
    if (p.S == 1) return launch(lc, kern, grid, block, smem, tm, a);
    return launch_cluster(lc, kern, grid, block, smem, dim3(p.S, 1, 1), tm, a);
}

template <bool XQ, bool ZEROS, int G>
cudaError_t run_rows(const Launch &lc, const W4Args &a, const uint8_t *codes) {
    if (a.M <= 8) return run_w4<XQ, ZEROS, G, 1>(lc, a, codes);
    if (a.M <= 16) return run_w4<XQ, ZEROS, G, 2>(lc, a, codes);
    return run_w4<XQ, ZEROS, G, 4>(lc, a, codes);
}

template <bool XQ, bool ZEROS>
cudaError_t run_group(const Launch &lc, const W4Args &a, const uint8_t *codes, int group) {
    switch (group) {
        case 32: return run_rows<XQ, ZEROS, 32>(lc, a, codes);
        case 64: return run_rows<XQ, ZEROS, 64>(lc, a, codes);
        case 128: return run_rows<XQ, ZEROS, 128>(lc, a, codes);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

W4Plan plan_gemv_w4(int num_sms, int M, int K, int N, int group, bool zeros) {
    const int m = M < pass_rows(K) ? M : pass_rows(K);
    switch (group) {
        case 32: return zeros ? plan_rows<true, 32>(num_sms, m, K, N) : plan_rows<false, 32>(num_sms, m, K, N);
        case 64: return zeros ? plan_rows<true, 64>(num_sms, m, K, N) : plan_rows<false, 64>(num_sms, m, K, N);
        default: return zeros ? plan_rows<true, 128>(num_sms, m, K, N) : plan_rows<false, 128>(num_sms, m, K, N);
    }
}

cudaError_t launch_gemv_w4(const Launch &lc, const void *x, const float *xs, int M, int K, const uint8_t *codes,
                           const bf16 *scales, const uint8_t *zeros, int group, int N, int epi, void *out) {
    const int pass = pass_rows(K);
    for (int m0 = 0; m0 < M; m0 += pass) {
        W4Args a = {};
        a.M = M - m0 < pass ? M - m0 : pass;
        a.K = K;
        a.N = N;
        a.x = static_cast<const uint8_t *>(x) + (size_t)m0 * K * (xs ? 1 : 2);
        a.xs = xs ? xs + m0 : nullptr;
        a.scales = scales;
        a.zeros = zeros;
        a.out = static_cast<uint8_t *>(out) + (size_t)m0 * N * (epi == EPI_SWIGLU ? 1 : 4);
        a.epi = epi;
        a.limit = lc.wait_limit;
        const cudaError_t e = xs ? (zeros ? run_group<true, true>(lc, a, codes, group) : run_group<true, false>(lc, a, codes, group))
                                 : (zeros ? run_group<false, true>(lc, a, codes, group) : run_group<false, false>(lc, a, codes, group));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace q3
