// C ABI of the single kernels on 8-bit and 4-bit operands: argument checks and launches.  See
// include/qwen3_gb300.h for the contract of every call.

#include <atomic>
#include <cmath>
#include <string>

#include "kernels.h"
#include "qwen3_gb300.h"

namespace q3 {
void set_last_error(const std::string &msg);  // message returned by qwen3_last_error(NULL)
}

namespace {

using namespace q3;

int fail(int code, const char *call, const char *why) {
    set_last_error(std::string(call) + ": " + why);
    return code;
}

int done(cudaError_t e, const char *call) {
    return e == cudaSuccess ? QWEN3_OK : fail(QWEN3_E_CUDA, call, cudaGetErrorString(e));
}

bool aligned16(const void *a, const void *b = nullptr, const void *c = nullptr, const void *d = nullptr) {
    return !((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c) |
              reinterpret_cast<uintptr_t>(d)) & 15);
}

bool misaligned(const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to; }

bool dtype_ok(int32_t t) { return t == QWEN3_DT_F32 || t == QWEN3_DT_BF16; }

constexpr int32_t MAX_SIZE = 1 << 30;  // rows or columns: sums with a tile stay in 32 bits

std::atomic<uint32_t> wait_limit_cycles{0};  // 0: the default

cudaError_t make_launch(void *stream, Launch *lc) {
    lc->stream = static_cast<cudaStream_t>(stream);
    if (const uint32_t cycles = wait_limit_cycles.load(std::memory_order_relaxed)) lc->wait_limit = cycles;
    // Every kernel here touches memory only after the one before it in the stream is done, and then lets
    // the next one launch, whose start hides behind it (back to back from Python: 13 rows of 8192 x
    // 10240 25.8 -> 23.4 us then, 23,460 rows quantised 28.9 -> 25.6; in a graph one row of q/k/v 3.9 -> 3.3).
    lc->pdl = true;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return cudaDeviceGetAttribute(&lc->num_sms, cudaDevAttrMultiProcessorCount, dev);
}

// Runs an entry point's body; an exception (an allocation of the host that failed) becomes a code.
template <typename F>
int guarded(F body) noexcept {
    try {
        set_last_error("");
        return body();
    } catch (...) {
        return QWEN3_E_CUDA;
    }
}

}  // namespace

extern "C" {

void qwen3_op_set_wait_limit(uint32_t cycles) { wait_limit_cycles.store(cycles, std::memory_order_relaxed); }

int qwen3_op_quant_q8(const void *x, int32_t x_dtype, int32_t M, int32_t K, void *q, float *scale, void *stream) {
    return guarded([&]() -> int {
        const char *call = "qwen3_op_quant_q8";
        if (!x || !q || !scale) return fail(QWEN3_E_INVALID, call, "NULL argument");
        if (M < 1 || M > MAX_SIZE || !rows_q8_supported(K))
            return fail(QWEN3_E_INVALID, call, "bad size (K a multiple of 16 from 16 to 16384)");
        if (!dtype_ok(x_dtype)) return fail(QWEN3_E_INVALID, call, "x_dtype must be QWEN3_DT_F32 or QWEN3_DT_BF16");
        if (misaligned(x, 32) || !aligned16(q) || misaligned(scale, 4))
            return fail(QWEN3_E_INVALID, call, "x must be 32-byte aligned, q 16 (scale 4)");
        Launch lc;
        cudaError_t e = make_launch(stream, &lc);
        if (e == cudaSuccess) e = launch_quant_q8(lc, x, x_dtype == QWEN3_DT_BF16, M, K, static_cast<uint8_t *>(q), scale);
        return done(e, call);
    });
}

int qwen3_op_add_rmsnorm_q8(float *h, const void *delta, int32_t delta_dtype, int32_t M, int32_t C, const float *gain,
                            float eps, void *q, float *scale, void *stream) {
    return guarded([&]() -> int {
        const char *call = "qwen3_op_add_rmsnorm_q8";
        if (!h || !gain || !q || !scale) return fail(QWEN3_E_INVALID, call, "NULL argument");
        if (M < 1 || M > MAX_SIZE || !rows_q8_supported(C))
            return fail(QWEN3_E_INVALID, call, "bad size (C a multiple of 16 from 16 to 16384)");
        if (delta && !dtype_ok(delta_dtype))
            return fail(QWEN3_E_INVALID, call, "delta_dtype must be QWEN3_DT_F32 or QWEN3_DT_BF16");
        if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(QWEN3_E_INVALID, call, "eps must be finite and >= 0");
        if (misaligned(h, 32) || misaligned(delta, 32) || !aligned16(gain, q) || misaligned(scale, 4))
            return fail(QWEN3_E_INVALID, call, "h and delta must be 32-byte aligned, gain and q 16 (scale 4)");
        Launch lc;
        cudaError_t e = make_launch(stream, &lc);
        if (e == cudaSuccess)
            e = launch_add_rmsnorm_q8(lc, h, delta, delta_dtype == QWEN3_DT_BF16, M, C, gain, eps, static_cast<uint8_t *>(q),
                                      scale);
        return done(e, call);
    });
}

static bool gemm_q8_size(int32_t M, int32_t K, int32_t N) {
    return M >= 1 && M <= MAX_SIZE && N >= 16 && N <= MAX_SIZE && N % 16 == 0 && K >= 16 && K <= MAX_SIZE && K % 16 == 0;
}

int qwen3_op_gemm_q8_plan(int32_t M, int32_t K, int32_t N, int32_t *tile_cols, int32_t *k_shares) {
    return guarded([&]() -> int {
        const char *call = "qwen3_op_gemm_q8_plan";
        if (!tile_cols || !k_shares) return fail(QWEN3_E_INVALID, call, "NULL argument");
        if (!gemm_q8_size(M, K, N)) return fail(QWEN3_E_INVALID, call, "bad size (N and K multiples of 16)");
        Launch lc;
        const cudaError_t e = make_launch(nullptr, &lc);
        if (e != cudaSuccess) return done(e, call);
        const Q8Plan p = plan_gemm_q8(lc.num_sms, M, K, N);
        *tile_cols = p.tile_cols;
        *k_shares = p.k_shares;
        return QWEN3_OK;
    });
}

int qwen3_op_gemm_q8(const void *xq, const float *xs, int32_t M, int32_t K, const void *wq, const float *ws, int32_t N,
                     int32_t epi, void *out, void *stream) {
    return guarded([&]() -> int {
        const char *call = "qwen3_op_gemm_q8";
        if (!xq || !xs || !wq || !ws || !out) return fail(QWEN3_E_INVALID, call, "NULL argument");
        if (!gemm_q8_size(M, K, N))
            return fail(QWEN3_E_INVALID, call, "bad size (N and K multiples of 16)");
        if (epi < QWEN3_EPI_F32 || epi > QWEN3_EPI_SWIGLU) return fail(QWEN3_E_INVALID, call, "unknown epilogue");
        if (!aligned16(xq, wq, ws, out) || misaligned(xs, 4))
            return fail(QWEN3_E_INVALID, call, "xq, wq, ws and out must be 16-byte aligned (xs 4)");
        Launch lc;
        cudaError_t e = make_launch(stream, &lc);
        if (e == cudaSuccess)
            e = launch_gemm_q8(lc, static_cast<const uint8_t *>(xq), xs, M, K, static_cast<const uint8_t *>(wq), ws, N, epi, out);
        return done(e, call);
    });
}

int qwen3_op_quant_w4(const void *w, int32_t N, int32_t K, int32_t group, void *codes, void *scales, void *zeros,
                      void *stream) {
    return guarded([&]() -> int {
        const char *call = "qwen3_op_quant_w4";
        if (!w || !codes || !scales) return fail(QWEN3_E_INVALID, call, "NULL argument");
        if (group != 32 && group != 64 && group != 128) return fail(QWEN3_E_INVALID, call, "group must be 32, 64 or 128");
        if (N < 1 || N > MAX_SIZE || K < group || K > MAX_SIZE || K % group)
            return fail(QWEN3_E_INVALID, call, "bad size (K a multiple of group)");
        if ((long long)N * K / 8 > (1ll << 38)) return fail(QWEN3_E_INVALID, call, "bad size (more than 2^41 weights)");
        if (misaligned(w, 32) || !aligned16(codes) || misaligned(scales, 2))
            return fail(QWEN3_E_INVALID, call, "w must be 32-byte aligned, codes 16 (scales 2)");
        Launch lc;
        cudaError_t e = make_launch(stream, &lc);
        if (e == cudaSuccess)
            e = launch_quant_w4(lc, static_cast<const bf16 *>(w), N, K, group, static_cast<uint8_t *>(codes),
                                static_cast<bf16 *>(scales), static_cast<uint8_t *>(zeros));
        return done(e, call);
    });
}

static bool gemv_w4_size(int32_t M, int32_t K, int32_t group, int32_t N) {
    return M >= 1 && M <= MAX_SIZE && N >= 1 && N <= MAX_SIZE && K >= group && K <= 65536 && K % group == 0;
}

int qwen3_op_gemv_w4_plan(int32_t M, int32_t K, int32_t group, int32_t with_zeros, int32_t N, int32_t *warps,
                          int32_t *col_shares, int32_t *cluster, int32_t *rounds) {
    return guarded([&]() -> int {
        const char *call = "qwen3_op_gemv_w4_plan";
        if (!warps || !col_shares || !cluster || !rounds) return fail(QWEN3_E_INVALID, call, "NULL argument");
        if (group != 32 && group != 64 && group != 128) return fail(QWEN3_E_INVALID, call, "group must be 32, 64 or 128");
        if (!gemv_w4_size(M, K, group, N)) return fail(QWEN3_E_INVALID, call, "bad size (K a multiple of group, at most 65536)");
        Launch lc;
        const cudaError_t e = make_launch(nullptr, &lc);
        if (e != cudaSuccess) return done(e, call);
        const W4Plan p = plan_gemv_w4(lc.num_sms, M, K, N, group, with_zeros != 0);
        *warps = p.NW;
        *col_shares = p.WK;
        *cluster = p.S;
        *rounds = p.rounds;
        return QWEN3_OK;
    });
}

int qwen3_op_gemv_w4(const void *x, const float *xs, int32_t M, int32_t K, const void *codes, const void *scales,
                     const void *zeros, int32_t group, int32_t N, int32_t epi, void *out, void *stream) {
    return guarded([&]() -> int {
        const char *call = "qwen3_op_gemv_w4";
        if (!x || !codes || !scales || !out) return fail(QWEN3_E_INVALID, call, "NULL argument");
        if (group != 32 && group != 64 && group != 128) return fail(QWEN3_E_INVALID, call, "group must be 32, 64 or 128");
        if (epi < QWEN3_EPI_F32 || epi > QWEN3_EPI_SWIGLU) return fail(QWEN3_E_INVALID, call, "unknown epilogue");
        if (!gemv_w4_size(M, K, group, N) || (epi == QWEN3_EPI_SWIGLU && N % 2))
            return fail(QWEN3_E_INVALID, call, "bad size (K a multiple of group, at most 65536; N even with SwiGLU)");
        if (!aligned16(x, codes, out) || misaligned(xs, 4) || misaligned(scales, 4) || misaligned(zeros, 4))
            return fail(QWEN3_E_INVALID, call, "x, codes and out must be 16-byte aligned (xs, scales and zeros 4)");
        Launch lc;
        cudaError_t e = make_launch(stream, &lc);
        if (e == cudaSuccess)
            e = launch_gemv_w4(lc, x, xs, M, K, static_cast<const uint8_t *>(codes), static_cast<const bf16 *>(scales),
                               static_cast<const uint8_t *>(zeros), group, N, epi, out);
        return done(e, call);
    });
}

}  // extern "C"
