// Quantisers: rows into e4m3 codes with one fp32 scale each, alone or after the residual add and
// RMSNorm (k_rows_q8, k_rows_q8_bf16), and weight groups into 4-bit codes (k_quant_w4).
//
// 8-bit rows.  scale = max|y| / 448 (448 the largest e4m3 value), code = e4m3(448 y / max|y|).
// For RMSNorm y_i = h_i r g_i with r = rsqrt(mean h^2 + eps) the factor r cancels out of the
// codes, so the sum of squares and the maximum of |h g| are reductions over the same loads and
// the row is read once: it stays in registers between the reductions and the codes.
// The quotient 448 y / m is q0 + (448 y - q0 m) / m with q0 = 448 y * (1 / m) and the remainder
// exact by FMA (Markstein's correction of an approximate quotient), so that quotients that
// are ties between two codes -- common for bf16 rows, whose 448 y is exact -- round to even
// as the definition says and do not depend on the error of 1 / m.  fp32 rows, whose 448 y rounds,
// take their quotient as a sum of two floats, so that every code is the nearest (exact_quotient).
// Bound by HBM: 3 to 13 bytes an element.  A row's warps hold it whole, 32 bytes a load, so that each
// byte moves once: 23,460 rows of 1,024 with a bf16 addend (264 MB) in 45.0 us, 5.9 TB/s, where a
// copy of as many bytes takes 41.5; 23,460 bf16 rows of 2,048 (144 MB) in 25.3 us.  With 16-byte
// loads the first took 48.3.

#include <cuda_fp8.h>

#include <type_traits>

#include "kernels.h"

namespace q3 {

namespace {

constexpr int ROW_PER_LANE = 4;                      // eight elements of a row held by one lane, times
constexpr int ROW_PER_WARP = ROW_PER_LANE * 32 * 8;  // 1,024 elements

// 32 bytes, read once.
__device__ __forceinline__ void load32(const void *p, uint32_t *u) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void store32(void *p, const float *v) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                 "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

// The i-th eight elements.
__device__ __forceinline__ void load8(const float *p, size_t i, float *v) {
    uint32_t u[8];
    load32(p + i * 8, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(u[e]);
}
__device__ __forceinline__ void load8(const bf16 *p, size_t i, float *v) { unpack8(ld_stream(p + i * 8), v); }

// max(m, |x|), NaN if either is.
__device__ __forceinline__ float max_abs(float m, float x) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(x)));
    return r;
}

// Reductions over the W warps of a row, in the same order in each of them.  Bit patterns of
// non-negative floats order like the floats, NaN above all.
template <int W, bool SUM>
__device__ __forceinline__ void row_reduce(float &ss, uint32_t &top, float *red_s, uint32_t *red_m) {
    if (SUM) ss = warp_sum(ss);
    top = __reduce_max_sync(0xffffffffu, top);
    if (W > 1) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) {
            if (SUM) red_s[warp] = ss;
            red_m[warp] = top;
        }
        __syncthreads();
        const int w0 = warp / W * W;
        ss = 0.0f;
        top = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (SUM) ss += red_s[w0 + w];
            top = max(top, red_m[w0 + w]);
        }
    }
}

// Packed fp32 arithmetic: two values an instruction.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// How a row's values become codes: code = e4m3((y k) / m) with m = max|y| pre, k = 448 pre.  A row
// that is not finite has k NaN, and so NaN codes; a row of zeros has inv 0, and so codes 0.
struct RowCode {
    float m, k, inv, pre;
    bool bad, zero;
};

__device__ __forceinline__ RowCode row_code(uint32_t top, bool bad) {
    RowCode c;
    const float amax = __uint_as_float(top);
    c.bad = bad || top >= 0x7f800000u;
    c.zero = top == 0;
    // a power of two that keeps 448 y, m and 1 / m normal numbers
    const float pre = amax < 0x1p-60f ? 0x1p+80f : amax > 0x1p+60f ? 0x1p-60f : 1.0f;
    c.m = c.zero ? 1.0f : amax * pre;
    c.pre = c.bad ? __uint_as_float(0x7fffffffu) : pre;
    c.k = Q8_MAX * c.pre;
    c.inv = c.zero ? 0.0f : 1.0f / c.m;
    return c;
}

__device__ __forceinline__ float2 quotients(float y0, float y1, const RowCode &c) {
    const uint64_t inv = pack2(c.inv, c.inv), n = mul2(pack2(y0, y1), pack2(c.k, c.k)), q = mul2(n, inv);
    return unpack2(fma2(fma2(q, pack2(-c.m, -c.m), n), inv, q));
}

// 448 y / m for any fp32 y, rounded so that its nearest e4m3 value is that of the exact quotient.
// h is y / m to an ulp with remainder r, exact by FMA; 448 h + 448 r / m is summed to s + e with
// |e| at most half an ulp of s.  Between two codes' tie and s lies a float unless s is the tie:
// only values of few bits can be ties, and those move by an ulp towards e.  448 y and a tie times m are
// integers of at most 33 bits in a common unit, so a quotient that is not a tie is 2^-33 of it
// away from one, and an |e| below 2^-40 is the error of this arithmetic (2^-46).
__device__ __forceinline__ float exact_quotient(float y, const RowCode &c) {
    const float v = y * c.pre;
    const float h = v * c.inv, r = fmaf(-h, c.m, v);
    const float p = h * Q8_MAX;
    const float t = fmaf(r * c.inv, Q8_MAX, fmaf(h, Q8_MAX, -p));
    const float s = p + t, e = t - (s - p);
    if ((__float_as_uint(s) & 0xfffu) || fabsf(e) <= fabsf(s) * 0x1p-40f) return s;
    return __uint_as_float(__float_as_uint(s) + ((e > 0.0f) == (s > 0.0f) ? 1u : ~0u));
}

// Whether a quotient of two roundings could lie on the other side of a tie than its exact value:
// within 4 ulp of a midpoint of e4m3's normal numbers, or among its subnormals, which are few.
__device__ __forceinline__ bool doubtful(float q) {
    const uint32_t b = __float_as_uint(q);
    return ((b - 0x7fffcu) & 0xfffffu) <= 8u || (fabsf(q) < 0x1p-6f && q != 0.0f);
}

// Four values as four e4m3 codes.
template <bool EXACT>
__device__ __forceinline__ uint32_t codes4(const float4 &y, const RowCode &c) {
    float2 a = quotients(y.x, y.y, c), b = quotients(y.z, y.w, c);
    if (EXACT && (doubtful(a.x) || doubtful(a.y) || doubtful(b.x) || doubtful(b.y))) {
        a = make_float2(exact_quotient(y.x, c), exact_quotient(y.y, c));
        b = make_float2(exact_quotient(y.z, c), exact_quotient(y.w, c));
    }
    return (uint32_t)__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16;
}

// Warps of a CTA whose rows take W warps each: small CTAs, so that the last ones end together (2%
// against 8 warps to a CTA).
constexpr int cta_warps(int W) { return W <= 4 ? 4 : W; }

// W warps to a row.  NORM: h is the residual and T the addend's type (HAS_D); else T is fp32,
// the input's type.  TINY: eps is below 2^-90, so that the squares of a tiny row count although they are below fp32's
// normal numbers (a kernel of its own: as a branch of the other it took 23,460 rows of 1,024 from 45.7 to 49.9 us).
template <typename T, bool NORM, bool HAS_D, bool TINY, int W>
__global__ void __launch_bounds__(cta_warps(W) * 32) k_rows_q8(const T *__restrict__ x, float *__restrict__ h,
                                                             const float *__restrict__ gain, int M, int C, float eps,
                                                             uint8_t *__restrict__ q, float *__restrict__ scale) {
    constexpr int WARPS = cta_warps(W);
    constexpr int PER = W == 32 ? 2 : ROW_PER_LANE;  // the longest rows hold 16 elements a lane of 32 warps
    __shared__ float red_s[WARPS];
    __shared__ uint32_t red_m[WARPS];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x * (WARPS / W) + warp / W;
    const bool live = row < M;  // the row's warps share a CTA-wide barrier with the others'
    const int c8 = C / 8, first = (warp % W) * 32 + lane;
    const size_t base = (size_t)row * c8;
    float v[PER][8], d[NORM && HAS_D ? PER : 1][8];
    float ss = 0.0f, most = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = first + j * W * 32;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = 0.0f;
        if (live && i < c8) {
            if (NORM)
                load8(h, base + i, v[j]);
            else
                load8(x, base + i, v[j]);
            if (NORM && HAS_D) load8(x, base + i, d[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = first + j * W * 32;
        if (NORM && HAS_D && live && i < c8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] += d[j][e];
            store32(h + (base + i) * 8, v[j]);
        }
        if (NORM && i < c8) {
            const float4 *gp = reinterpret_cast<const float4 *>(gain) + 2 * i;
            const float4 g0 = __ldg(gp), g1 = __ldg(gp + 1);
            const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss += v[j][e] * v[j][e];
                v[j][e] *= g[e];
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) most = max_abs(most, v[j][e]);
    }
    uint32_t top = __float_as_uint(most);
    row_reduce<W, NORM>(ss, top, red_s, red_m);
    float small = 0.0f;  // the squares' sum times 2^200, from the row as it is in memory now (this thread's own stores)
    if (TINY) {
        if (live)
            for (int i = first; i < c8; i += W * 32) {
                float y[8];
                load8(h, base + i, y);
#pragma unroll
                for (int e = 0; e < 8; ++e) small += (y[e] * 0x1p100f) * (y[e] * 0x1p100f);
            }
        uint32_t none = 0;
        if (W > 1) __syncthreads();  // the reduction before has been read
        row_reduce<W, true>(small, none, red_s, red_m);
    }
    if (!live) return;
    const RowCode c = row_code(top, NORM && !(ss < __uint_as_float(0x7f800000u)));
    if (warp % W == 0 && lane == 0) {
        float s = __uint_as_float(top);
        if (TINY && ss < 0x1p-100f)
            s = s * 0x1p100f * (1.0f / sqrtf(small / (float)C + eps * 0x1p100f * 0x1p100f));
        else if (NORM)
            s *= 1.0f / sqrtf(ss / (float)C + eps);
        scale[row] = c.bad ? __uint_as_float(0x7fffffffu) : c.zero ? 0.0f : s / Q8_MAX;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = first + j * W * 32;
        const float *y = v[j];
        if (i < c8)
            __stcs(reinterpret_cast<uint2 *>(q) + base + i,
                   make_uint2(codes4<!NORM>(make_float4(y[0], y[1], y[2], y[3]), c),
                              codes4<!NORM>(make_float4(y[4], y[5], y[6], y[7]), c)));
    }
}

// bf16 rows stay packed between the maximum and the codes: 64 elements to a lane, 2,048 to a warp.
constexpr int BF_PER_LANE = 4;  // 32-byte pieces
constexpr int BF_PER_WARP = BF_PER_LANE * 32 * 16;

template <int W>
__global__ void __launch_bounds__(cta_warps(W) * 32) k_rows_q8_bf16(const bf16 *__restrict__ x, int M, int K,
                                                                  uint8_t *__restrict__ q, float *__restrict__ scale) {
    constexpr int WARPS = cta_warps(W), PER = W == 32 ? 1 : BF_PER_LANE;
    __shared__ uint32_t red_m[WARPS];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x * (WARPS / W) + warp / W;
    const bool live = row < M;
    const int k16 = K / 16, first = (warp % W) * 32 + lane;
    const size_t base = (size_t)row * k16;
    uint32_t v[PER][8];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = first + j * W * 32;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = 0;
        if (live && i < k16) load32(x + (base + i) * 16, v[j]);
    }
    __nv_bfloat162 most = __float2bfloat162_rn(0.0f);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(v[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) most = __hmax2_nan(most, __habs2(p[e]));
    }
    uint32_t top = max(__float_as_uint(__low2float(most)), __float_as_uint(__high2float(most)));
    float none = 0.0f;
    row_reduce<W, false>(none, top, nullptr, red_m);
    if (!live) return;
    const RowCode c = row_code(top, false);
    if (warp % W == 0 && lane == 0)
        scale[row] = c.bad ? __uint_as_float(0x7fffffffu) : __uint_as_float(top) / Q8_MAX;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = first + j * W * 32;
        if (i < k16) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t a = v[j][2 * e], b = v[j][2 * e + 1];
                o[e] = codes4<false>(make_float4(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u),
                                                 __uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u)),
                                     c);
            }
            __stcs(reinterpret_cast<uint4 *>(q) + base + i, make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
}

// W warps to a row for rows of `warps` warps' worth: no more than hold it, so that a lane has its
// four loads in flight, but up to 32 where there are few rows, two to an SM at most, and the time is one row's
// latency (5 rows of 1,024: 2.0 us with one load a lane, 3.0 with four).
template <typename Go>
cudaError_t by_warps(const Launch &lc, int M, int warps, Go go) {
    if (M <= 2 * lc.num_sms) warps = warps * 4 < 32 ? warps * 4 : 32;
    if (warps <= 1) return go(std::integral_constant<int, 1>());
    if (warps <= 2) return go(std::integral_constant<int, 2>());
    if (warps <= 4) return go(std::integral_constant<int, 4>());
    if (warps <= 8) return go(std::integral_constant<int, 8>());
    if (warps <= 16) return go(std::integral_constant<int, 16>());
    return go(std::integral_constant<int, 32>());
}

dim3 row_grid(int M, int W) {
    const int rows = cta_warps(W) / W;
    return dim3((unsigned)(((long long)M + rows - 1) / rows));
}

template <typename T, bool NORM, bool HAS_D, bool TINY = false>
cudaError_t run_rows(const Launch &lc, const T *x, float *h, const float *gain, int M, int C, float eps, uint8_t *q,
                     float *scale) {
    if constexpr (NORM && !TINY)
        if (eps < 0x1p-90f) return run_rows<T, NORM, HAS_D, true>(lc, x, h, gain, M, C, eps, q, scale);
    return by_warps(lc, M, (C + ROW_PER_WARP - 1) / ROW_PER_WARP, [&](auto w) {
        constexpr int W = decltype(w)::value;
        return launch(lc, k_rows_q8<T, NORM, HAS_D, TINY, W>, row_grid(M, W), dim3(cta_warps(W) * 32), 0, x, h, gain, M, C, eps, q,
                      scale);
    });
}

// ---- 4-bit weights --------------------------------------------------------------------------
//
// Sixteen weights (32 bytes) to a lane, so a group of G is G / 16 neighbouring lanes whose extremes
// meet by shuffles; each lane writes its 8 bytes of codes.  The scale is rounded to bf16 before the
// codes are taken from it, so they match the scale that is stored.
//   The quotients w / s must round as the definition's do, and between bf16 numbers that is only in
// doubt at exact ties (other quotients are 2^-17 or more away from one): Markstein's correction
// makes those exact at three instructions for two weights (packed fp32) where a division takes a
// dozen for one.  The head's 155 M weights in groups of 32 with zero points (405 MB): 165 us with
// divisions, issue-bound; 64 us now, 6.3 TB/s.  Ranges outside [2^-95, 2^95] take the divisions.

// x / d for a constant d, correctly rounded (x normal, the quotient far from underflow).
__device__ __forceinline__ float over(float x, float d, float inv) {
    const float q = x * inv;
    return fmaf(fmaf(-q, d, x), inv, q);
}

template <int G, bool ZEROS>
__global__ void __launch_bounds__(256) k_quant_w4(const bf16 *__restrict__ w, long long n16, uint2 *__restrict__ codes,
                                                  bf16 *__restrict__ scales, uint8_t *__restrict__ zeros) {
    constexpr int LANES = G / 16;
    pdl_wait();
    pdl_trigger();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;  // n16 is a multiple of LANES
    const bool live = i < n16;
    uint32_t u[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (live) load32(w + i * 16, u);
    const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(u);
    // extremes, in bf16 pairs; a NaN carries through
    __nv_bfloat162 lo = __float2bfloat162_rn(0.0f), hi = lo;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (ZEROS) {
            lo = __hmin2_nan(lo, p[j]);
            hi = __hmax2_nan(hi, p[j]);
        } else {
            hi = __hmax2_nan(hi, __habs2(p[j]));
        }
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        if (ZEROS) lo = __hmin2_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = __hmax2_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (!live) return;
    const bf16 l = __hmin_nan(__low2bfloat16(lo), __high2bfloat16(lo)), m = __hmax_nan(__low2bfloat16(hi), __high2bfloat16(hi));
    const float least = __bfloat162float(l), range = ZEROS ? __bfloat162float(m) - least : __bfloat162float(m);
    const bool usual = range > 0x1p-95f && range < 0x1p+95f;  // false for a NaN
    bf16 sb;
    float z = 8.0f;
    uint32_t c[2] = {0, 0};
    if (usual) {
        sb = __float2bfloat16(ZEROS ? over(range, 15.0f, 1.0f / 15.0f) : over(range, 7.0f, 1.0f / 7.0f));
        const float s = __bfloat162float(sb), inv = __fdividef(1.0f, s);
        // the integer nearest to y (ties to even), |y| < 2^21, is the low bits of y + 1.5 2^23
        const int zi = ZEROS ? __float_as_int(over(-least, s, inv) + 12582912.0f) - 0x4b400000 : 8;  // at most rint(15 (1 + 2^-8))
        z = (float)zi;
        const uint64_t inv2 = pack2(inv, inv), s2 = pack2(-s, -s), magic = pack2(12582912.0f, 12582912.0f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint64_t x = pack2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u));
            const uint64_t q = mul2(x, inv2);
            const float2 t = unpack2(add2(fma2(fma2(q, s2, x), inv2, q), magic));
            // within [0, 16]: |w| <= 7 s (1 + 2^-8), or w - least <= 15 s (1 + 2^-8) and both ends round
            int v0 = __float_as_int(t.x) + (zi - 0x4b400000), v1 = __float_as_int(t.y) + (zi - 0x4b400000);
            if (ZEROS) {
                v0 = min(v0, 15);
                v1 = min(v1, 15);
            }
            c[j / 4] += (uint32_t)v0 << (8 * (j & 3));
            c[j / 4] += (uint32_t)v1 << (8 * (j & 3) + 4);
        }
    } else {  // as the definition says, step by step
        float step = ZEROS ? range / 15.0f : range / 7.0f;
        if (ZEROS && range > 3.4e38f)  // finite ends whose distance is past fp32: at a sixteenth of its size
            step = (__bfloat162float(m) * 0.0625f - least * 0.0625f) / 15.0f * 16.0f;
        sb = __float2bfloat16(step);
        const float s = __bfloat162float(sb);
        const bool bad = !(s <= 3.4e38f);  // a group that is not finite
        const float div = bad || !(s > 0.0f) ? 1.0f : s;
        if (ZEROS) z = bad ? 0.0f : fminf(fmaxf(rintf(-least / div), 0.0f), 15.0f);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const uint32_t bits = j & 1 ? u[j / 2] & 0xffff0000u : u[j / 2] << 16;
            const float r = bad ? z : fminf(fmaxf(rintf(__uint_as_float(bits) / div) + z, 0.0f), 15.0f);
            c[j / 8] += (uint32_t)(int)r << (4 * (j & 7));
        }
        if (bad) sb = __ushort_as_bfloat16(0x7fff);
    }
    __stcs(codes + i, make_uint2(c[0], c[1]));
    if ((threadIdx.x & (LANES - 1)) == 0) {
        scales[i / LANES] = sb;
        if (ZEROS) zeros[i / LANES] = (uint8_t)(int)z;
    }
}

}  // namespace

bool rows_q8_supported(int C) { return C >= 16 && C % 16 == 0 && C <= 16 * ROW_PER_WARP; }

cudaError_t launch_quant_q8(const Launch &lc, const void *x, bool x_bf16, int M, int K, uint8_t *q, float *scale) {
    if (x_bf16)
        return by_warps(lc, M, (K + BF_PER_WARP - 1) / BF_PER_WARP, [&](auto w) {
            constexpr int W = decltype(w)::value;
            return launch(lc, k_rows_q8_bf16<W>, row_grid(M, W), dim3(cta_warps(W) * 32), 0, (const bf16 *)x, M, K, q, scale);
        });
    return run_rows<float, false, false>(lc, (const float *)x, nullptr, nullptr, M, K, 0.0f, q, scale);
}

cudaError_t launch_add_rmsnorm_q8(const Launch &lc, float *h, const void *delta, bool delta_bf16, int M, int C,
                                  const float *gain, float eps, uint8_t *q, float *scale) {
    if (!delta) return run_rows<float, true, false>(lc, nullptr, h, gain, M, C, eps, q, scale);
    if (delta_bf16) return run_rows<bf16, true, true>(lc, (const bf16 *)delta, h, gain, M, C, eps, q, scale);
    return run_rows<float, true, true>(lc, (const float *)delta, h, gain, M, C, eps, q, scale);
}

cudaError_t launch_quant_w4(const Launch &lc, const bf16 *w, int N, int K, int group, uint8_t *codes, bf16 *scales,
                            uint8_t *zeros) {
    const long long n16 = (long long)N * K / 16;
    const long long blocks = (n16 + 255) / 256;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    auto go = [&](auto kern) {
        return launch(lc, kern, dim3((unsigned)blocks), dim3(256), 0, w, n16, reinterpret_cast<uint2 *>(codes), scales, zeros);
    };
    switch (group) {
        case 32: return zeros ? go(k_quant_w4<32, true>) : go(k_quant_w4<32, false>);
        case 64: return zeros ? go(k_quant_w4<64, true>) : go(k_quant_w4<64, false>);
        case 128: return zeros ? go(k_quant_w4<128, true>) : go(k_quant_w4<128, false>);
    }
    return cudaErrorInvalidValue;
}

}  // namespace q3
