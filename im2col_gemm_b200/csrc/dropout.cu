// dropout.cu -- dropout whose mask is drawn again wherever it is needed
// (include/mqc.h: mqc_dropout_fwd, mqc_dropout_bwd).
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "dense.cuh"
#include "host.h"

namespace mqc {
namespace {

// Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2,
// 3", SC 2011): ten rounds of two 32 x 32 -> 64-bit products.  The 64-bit
// variant that the stochastic quantizer uses would cost about twice the
// instructions per random bit here, and this pass is close to issue-bound.
// keys: the ten rounds' keys, advanced on the host.
struct PhiloxKeys {
    uint32_t k[10][2];
};
__device__ __forceinline__ uint4 philox4x32_10(uint4 c, const PhiloxKeys &keys) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = static_cast<uint64_t>(c.x) * 0xD2511F53u, q = static_cast<uint64_t>(c.z) * 0xCD9E8D57u;
        c = make_uint4(static_cast<uint32_t>(q >> 32) ^ c.y ^ keys.k[r][0], static_cast<uint32_t>(q),
                       static_cast<uint32_t>(p >> 32) ^ c.w ^ keys.k[r][1], static_cast<uint32_t>(p));
    }
    return c;
}

struct DropoutParams {
    const void *x, *res;
    void *y;
    int64_t ldx, ldr, ldy, cols, total;   // total = rows * cols
    uint64_t offset;
    const uint64_t *offset_dev;
    PhiloxKeys keys;
    uint32_t bar;                         // t << 16: an element stays when its 16 bits << 16 are >= bar
    int32_t none;                         // t = 65536: nothing stays
    float scale;
};

// Whether element e of a block stays: its half of the word, moved to the top,
// against the bar (the low bits under it decide nothing).
__device__ __forceinline__ bool stays(const uint32_t (&w)[4], int e, const DropoutParams &P) {
    return ((e & 1) ? w[e / 2] : w[e / 2] << 16) >= P.bar && !P.none;
}

// A thread owns one Philox block: eight consecutive elements of the logical
// row-major matrix.  Where they are contiguous in every tensor and start at
// 16-byte boundaries (kFlat: one long row, kRows: rows of whole blocks) they
// move as vectors; a last, partial block and everything else (kAny) goes
// element by element.
// Bound by memory, with the issue slots close behind (the ten rounds' products
// fill the multiplier): 16384 x 2048 bf16 with a residual moves 201 MB in 32.3
// to 33.0 us, 6.1 to 6.2 TB/s.
enum DropoutForm { kAny = 0, kRows = 1, kFlat = 2 };
template <typename T, int FORM>
__global__ void __launch_bounds__(256) dropout_kernel(const __grid_constant__ DropoutParams P) {
    const uint64_t offset = P.offset + (P.offset_dev ? *P.offset_dev : 0);
    const int64_t blocks = (P.total + 7) / 8;
    const T *x = static_cast<const T *>(P.x), *res = static_cast<const T *>(P.res);
    T *y = static_cast<T *>(P.y);
    constexpr int n = Vec<T>::n;
    for (int64_t b = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; b < blocks;
         b += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t i0 = b * 8;
        int64_t row = 0, col = i0;
        if (FORM != kFlat && P.cols != P.total) {
            row = P.total <= 0xFFFFFFFFll ? static_cast<uint32_t>(i0) / static_cast<uint32_t>(P.cols) : i0 / P.cols;
            col = i0 - row * P.cols;
        }
        if (FORM != kAny && i0 + 8 <= P.total) {
            uint4 xv[8 / n], rv[8 / n];
#pragma unroll
            for (int v = 0; v < 8 / n; ++v) xv[v] = reinterpret_cast<const uint4 *>(x + row * P.ldx + col)[v];
            if (res)
#pragma unroll
                for (int v = 0; v < 8 / n; ++v) rv[v] = reinterpret_cast<const uint4 *>(res + row * P.ldr + col)[v];
            const uint4 r = philox4x32_10(make_uint4(static_cast<uint32_t>(b), static_cast<uint32_t>(b >> 32),
                                                     static_cast<uint32_t>(offset), static_cast<uint32_t>(offset >> 32)),
                                          P.keys);
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int v = 0; v < 8 / n; ++v) {
                float f[n], scale[n];
                Vec<T>::widen(xv[v], f);
#pragma unroll
                for (int q = 0; q < n; ++q) scale[q] = P.scale;
                mul_to(f, scale);
#pragma unroll
                for (int q = 0; q < n; ++q) f[q] = stays(w, v * n + q, P) ? f[q] : 0.f;
                if (res) {
                    float a[n];
                    Vec<T>::widen(rv[v], a);
                    add_to(f, a);
                }
                reinterpret_cast<uint4 *>(y + row * P.ldy + col)[v] = Vec<T>::narrow(f);
            }
            continue;
        }
        const uint4 r = philox4x32_10(make_uint4(static_cast<uint32_t>(b), static_cast<uint32_t>(b >> 32),
                                                 static_cast<uint32_t>(offset), static_cast<uint32_t>(offset >> 32)),
                                      P.keys);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (i0 + e < P.total) {
                float f = stays(w, e, P) ? to_f32(x[row * P.ldx + col]) * P.scale : 0.f;
                if (res) f += to_f32(res[row * P.ldr + col]);
                y[row * P.ldy + col] = from_f32<T>(f);
                if (++col == P.cols) {
                    col = 0;
                    ++row;
                }
            }
        }
    }
}

template <typename T>
void launch(const DropoutParams &p, DropoutForm form, int sms, cudaStream_t s) {
    const int64_t blocks = std::min<int64_t>(ceil_div(ceil_div(p.total, 8), 256), int64_t(sms) * 32);
    const unsigned grid = static_cast<unsigned>(blocks);
    if (form == kFlat) dropout_kernel<T, kFlat><<<grid, 256, 0, s>>>(p);
    else if (form == kRows) dropout_kernel<T, kRows><<<grid, 256, 0, s>>>(p);
    else dropout_kernel<T, kAny><<<grid, 256, 0, s>>>(p);
}

mqc_status dropout(const char *name, const void *x, int64_t ldx, const void *res, int64_t ldr, int64_t rows,
                   int64_t cols, int32_t dtype, double p, uint64_t seed, uint64_t offset, const uint64_t *offset_dev,
                   void *y, int64_t ldy, void *stream) {
    if (dtype != MQC_F32 && dtype != MQC_BF16 && dtype != MQC_F16) return fail(MQC_ERR_INVALID, "%s: bad dtype", name);
    if (rows < 0 || cols < 0) return fail(MQC_ERR_INVALID, "%s: negative extent", name);
    if (!(p >= 0.0 && p <= 1.0)) return fail(MQC_ERR_INVALID, "%s: p must be within [0, 1]", name);
    if (rows == 0 || cols == 0) return MQC_OK;
    if (x == nullptr || y == nullptr) return fail(MQC_ERR_INVALID, "%s: null tensor", name);
    const int64_t most = int64_t(1) << 40;
    if (cols > most || rows > most / cols) return fail(MQC_ERR_INVALID, "%s: tensor too large", name);
    if (ldx < cols || ldy < cols || (res && ldr < cols) || ldx > most || ldy > most || (res && ldr > most))
        return fail(MQC_ERR_INVALID, "%s: row stride out of range", name);
    if (!aligned16(x) || !aligned16(y) || (res && !aligned16(res)))
        return fail(MQC_ERR_ALIGNMENT, "%s: tensor not 16-byte aligned", name);
    if ((reinterpret_cast<uintptr_t>(offset_dev) & 7u) != 0)
        return fail(MQC_ERR_ALIGNMENT, "%s: offset_dev not 8-byte aligned", name);
    if (rows > 1 && ((y == x && ldx != ldy) || (res && y == res && ldr != ldy)))
        return fail(MQC_ERR_INVALID, "%s: an output in place needs its input's row stride", name);
    DeviceLimits d;
    mqc_status st = device_limits(&d);
    if (st != MQC_OK) return st;
    DropoutParams P{};
    P.x = x;
    P.res = res;
    P.y = y;
    P.ldx = ldx;
    P.ldr = ldr;
    P.ldy = ldy;
    P.cols = cols;
    P.total = rows * cols;
    for (uint32_t r = 0; r < 10; ++r) {
        P.keys.k[r][0] = static_cast<uint32_t>(seed) + r * 0x9E3779B9u;
        P.keys.k[r][1] = static_cast<uint32_t>(seed >> 32) + r * 0xBB67AE85u;
    }
    P.offset = offset;
    P.offset_dev = offset_dev;
    const uint32_t t = static_cast<uint32_t>(std::floor(p * 65536.0 + 0.5));
    P.none = t >= 65536u;
    P.bar = P.none ? 0u : t << 16;
    P.scale = P.none ? 0.f : 65536.f / static_cast<float>(65536u - t);
    // rows that follow one another are one long row
    const bool one = rows == 1 || (ldx == cols && ldy == cols && (!res || ldr == cols));
    if (one) P.cols = P.total;
    const int64_t per16 = 16 / dtype_bytes(dtype);
    const bool rows16 = cols % 8 == 0 && ldx % per16 == 0 && ldy % per16 == 0 && (!res || ldr % per16 == 0);
    const DropoutForm form = one ? kFlat : (rows16 ? kRows : kAny);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == MQC_F32) launch<float>(P, form, d.sms, s);
    else if (dtype == MQC_BF16) launch<__nv_bfloat16>(P, form, d.sms, s);
    else launch<__half>(P, form, d.sms, s);
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MQC_OK : cuda_fail(e, "dropout_kernel launch");
}

}  // namespace
}  // namespace mqc

extern "C" {

mqc_status mqc_dropout_fwd(const void *x, int64_t ldx, const void *residual, int64_t ldr, int64_t rows, int64_t cols,
                           int32_t dtype, double p, uint64_t seed, uint64_t offset, const uint64_t *offset_dev,
                           void *y, int64_t ldy, void *stream) {
    return mqc::dropout("dropout_fwd", x, ldx, residual, ldr, rows, cols, dtype, p, seed, offset, offset_dev, y, ldy,
                        stream);
}

mqc_status mqc_dropout_bwd(const void *g, int64_t ldg, int64_t rows, int64_t cols, int32_t dtype, double p,
                           uint64_t seed, uint64_t offset, const uint64_t *offset_dev, void *gx, int64_t ldgx,
                           void *stream) {
    return mqc::dropout("dropout_bwd", g, ldg, nullptr, 0, rows, cols, dtype, p, seed, offset, offset_dev, gx, ldgx,
                        stream);
}

}  // extern "C"
