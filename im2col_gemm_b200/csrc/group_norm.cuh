// group_norm.cuh -- group norm with an activation over channels-last tensors,
// forward and backward.
#pragma once

#include "common.cuh"
#include "dense.cuh"

namespace mqc {

// VEC consecutive elements (VEC * sizeof(T) = 2 .. 16 bytes) loaded or stored
// as one access, as floats.
template <int BYTES> struct RawOf;
template <> struct RawOf<2> { using type = uint16_t; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<16> { using type = uint4; };
template <typename T, int VEC>
struct Pack {
    using Raw = typename RawOf<VEC * sizeof(T)>::type;
    __device__ static __forceinline__ Raw load(const T *p) { return *reinterpret_cast<const Raw *>(p); }
    __device__ static __forceinline__ void widen(const Raw &r, float (&v)[VEC]) {
        const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
        for (int q = 0; q < VEC; ++q) v[q] = to_f32(e[q]);
    }
    __device__ static __forceinline__ void store(T *p, const float (&v)[VEC]) {
        Raw r;
        T *e = reinterpret_cast<T *>(&r);
#pragma unroll
        for (int q = 0; q < VEC; ++q) e[q] = from_f32<T>(v[q]);
        *reinterpret_cast<Raw *>(p) = r;
    }
};

struct GnTensor {
    const void *p;
    int64_t sn, sp;                      // element strides of images and pixels
};

struct GnParams {
    GnTensor x, g;                       // g: incoming gradient (backward)
    void *out;                           // y or gx
    int64_t on, op;
    const float *gamma, *beta;
    float *mean, *rstd;                  // [N][G]
    float *part;                         // [N][slabs][2][C]
    float *coef;                         // [N][G][2] (backward)
    float *ggamma, *gbeta;
    float eps;
    int32_t N, C, G, D, HW;
    int32_t slabs, slab;                 // pixels per slab
    int32_t tx, ty, col_blocks;          // threads along channel vectors and pixels; blocks along channels
    int32_t act;
    int32_t chunks, gpc, splits, iters;  // on-chip form: channel chunks of gpc groups, CTAs of a cluster, slots a thread
};

constexpr int kGnThreads = 256;

// The block's image, pixel slab and channels, and this thread's place in it.
template <int VEC>
struct GnPlace {
    int n, slab, c, row, p0, p1;
    bool on;
    __device__ __forceinline__ explicit GnPlace(const GnParams &P) {
        int b = blockIdx.x;
        const int cb = b % P.col_blocks;
        b /= P.col_blocks;
        slab = b % P.slabs;
        n = b / P.slabs;
        row = threadIdx.x / P.tx;
        c = (cb * P.tx + threadIdx.x % P.tx) * VEC;
        on = row < P.ty && c < P.C;
        p0 = slab * P.slab + row;
        p1 = min(P.HW, (slab + 1) * P.slab);
    }
};

// Per channel and slab: mean and sum of squared deviations, by Welford's
// recurrence per thread (no difference of large squares), joined over the
// block's pixel rows in row order (Chan et al.).
template <typename T, int VEC>
__global__ void __launch_bounds__(kGnThreads) gn_stats_kernel(const __grid_constant__ GnParams P) {
    __shared__ float sh[2][kGnThreads * VEC];
    const GnPlace<VEC> at(P);
    float mean[VEC] = {}, m2[VEC] = {};
    if (at.on) {
        const T *x = static_cast<const T *>(P.x.p) + at.n * P.x.sn + at.c;
        float k = 0.f;
        constexpr int U = 4;
        for (int p = at.p0; p < at.p1; p += U * P.ty) {
            typename Pack<T, VEC>::Raw r[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p + u * P.ty < at.p1) r[u] = Pack<T, VEC>::load(x + (p + static_cast<int64_t>(u) * P.ty) * P.x.sp);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p + u * P.ty < at.p1) {
                    k += 1.f;
                    const float inv = __frcp_rn(k);
                    float v[VEC];
                    Pack<T, VEC>::widen(r[u], v);
#pragma unroll
                    for (int q = 0; q < VEC; ++q) {
                        const float d = v[q] - mean[q];
                        mean[q] += d * inv;
                        m2[q] += d * (v[q] - mean[q]);
                    }
                }
        }
    }
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
        sh[0][threadIdx.x * VEC + q] = mean[q];
        sh[1][threadIdx.x * VEC + q] = m2[q];
    }
    __syncthreads();
    // one thread per channel of the block; row t holds ceil((pixels - t) / ty)
    const int pixels = at.p1 - at.slab * P.slab, width = P.tx * VEC;
    const int c0 = (blockIdx.x % P.col_blocks) * width;
    for (int i = threadIdx.x; i < width && c0 + i < P.C; i += kGnThreads) {
        float n = 0.f, m = 0.f, s = 0.f;
        for (int t = 0; t < P.ty && t < pixels; ++t) {
            const float nt = static_cast<float>((pixels - t + P.ty - 1) / P.ty);
            const float d = sh[0][t * width + i] - m, tot = n + nt;
            m += d * (nt / tot);
            s += sh[1][t * width + i] + d * d * (n * nt / tot);
            n = tot;
        }
        float *out = P.part + (static_cast<int64_t>(at.n) * P.slabs + at.slab) * 2 * P.C + c0 + i;
        out[0] = m;
        out[P.C] = s;
    }
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// One warp per image and group: the partial statistics joined in double.
static __global__ void __launch_bounds__(128) gn_finish_kernel(const __grid_constant__ GnParams P) {
    const int64_t w = blockIdx.x * 4ll + threadIdx.x / 32;
    if (w >= static_cast<int64_t>(P.N) * P.G) return;
    const int lane = threadIdx.x % 32;
    const int n = static_cast<int>(w / P.G), g = static_cast<int>(w % P.G);
    const float *part = P.part + static_cast<int64_t>(n) * P.slabs * 2 * P.C + g * P.D;
    const int64_t entries = static_cast<int64_t>(P.slabs) * P.D;
    const double total = static_cast<double>(P.HW) * P.D;
    double sum = 0.0, dev = 0.0;
    for (int64_t e = lane; e < entries; e += 32) {
        const int s = static_cast<int>(e / P.D), c = static_cast<int>(e % P.D);
        const int cnt = min(P.HW, (s + 1) * P.slab) - s * P.slab;
        sum += cnt * static_cast<double>(part[static_cast<int64_t>(s) * 2 * P.C + c]);
    }
    const double mean = warp_sum(sum) / total;
    for (int64_t e = lane; e < entries; e += 32) {
        const int s = static_cast<int>(e / P.D), c = static_cast<int>(e % P.D);
        const int cnt = min(P.HW, (s + 1) * P.slab) - s * P.slab;
        const double d = part[static_cast<int64_t>(s) * 2 * P.C + c] - mean;
        dev += part[(static_cast<int64_t>(s) * 2 + 1) * P.C + c] + cnt * d * d;
    }
    dev = warp_sum(dev) / total;
    if (lane == 0) {
        P.mean[w] = static_cast<float>(mean);
        P.rstd[w] = static_cast<float>(1.0 / sqrt(dev + P.eps));
    }
}

// y = act((x - mean) (rstd gamma) + beta).
template <typename T, int VEC>
__global__ void __launch_bounds__(kGnThreads) gn_apply_kernel(const __grid_constant__ GnParams P) {
    const GnPlace<VEC> at(P);
    if (!at.on) return;
    float mean[VEC], a[VEC], b[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
        const int64_t s = static_cast<int64_t>(at.n) * P.G + (at.c + q) / P.D;
        mean[q] = P.mean[s];
        a[q] = P.rstd[s] * (P.gamma ? P.gamma[at.c + q] : 1.f);
        b[q] = P.beta ? P.beta[at.c + q] : 0.f;
    }
    const T *x = static_cast<const T *>(P.x.p) + at.n * P.x.sn + at.c;
    T *y = static_cast<T *>(P.out) + at.n * P.on + at.c;
    constexpr int U = 4;
    for (int p = at.p0; p < at.p1; p += U * P.ty) {
        typename Pack<T, VEC>::Raw r[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (p + u * P.ty < at.p1) r[u] = Pack<T, VEC>::load(x + (p + static_cast<int64_t>(u) * P.ty) * P.x.sp);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (p + u * P.ty < at.p1) {
                float v[VEC];
                Pack<T, VEC>::widen(r[u], v);
#pragma unroll
                for (int q = 0; q < VEC; ++q) v[q] = (v[q] - mean[q]) * a[q] + b[q];
                act_values(P.act, v);
                Pack<T, VEC>::store(y + (p + static_cast<int64_t>(u) * P.ty) * P.op, v);
            }
    }
}

// Per channel and slab: sums of dz and dz xhat.
template <typename T, int VEC>
__global__ void __launch_bounds__(kGnThreads) gn_bwd_sums_kernel(const __grid_constant__ GnParams P) {
    __shared__ float sh[2][kGnThreads * VEC];
    const GnPlace<VEC> at(P);
    float sa[VEC] = {}, sb[VEC] = {};
    if (at.on) {
        float mean[VEC], rstd[VEC], gamma[VEC], beta[VEC];
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
            const int64_t s = static_cast<int64_t>(at.n) * P.G + (at.c + q) / P.D;
            mean[q] = P.mean[s];
            rstd[q] = P.rstd[s];
            gamma[q] = P.gamma ? P.gamma[at.c + q] : 1.f;
            beta[q] = P.beta ? P.beta[at.c + q] : 0.f;
        }
        const T *x = static_cast<const T *>(P.x.p) + at.n * P.x.sn + at.c;
        const T *g = static_cast<const T *>(P.g.p) + at.n * P.g.sn + at.c;
        constexpr int U = 2;
        for (int p = at.p0; p < at.p1; p += U * P.ty) {
            typename Pack<T, VEC>::Raw rx[U], rg[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p + u * P.ty < at.p1) {
                    rx[u] = Pack<T, VEC>::load(x + (p + static_cast<int64_t>(u) * P.ty) * P.x.sp);
                    rg[u] = Pack<T, VEC>::load(g + (p + static_cast<int64_t>(u) * P.ty) * P.g.sp);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p + u * P.ty < at.p1) {
                    float xv[VEC], gv[VEC];
                    Pack<T, VEC>::widen(rx[u], xv);
                    Pack<T, VEC>::widen(rg[u], gv);
                    float z[VEC], sl[VEC];
#pragma unroll
                    for (int q = 0; q < VEC; ++q) {
                        xv[q] = (xv[q] - mean[q]) * rstd[q];
                        z[q] = xv[q] * gamma[q] + beta[q];
                    }
                    act_slopes(P.act, z, sl);
#pragma unroll
                    for (int q = 0; q < VEC; ++q) {
                        const float dz = gv[q] * sl[q];
                        sa[q] += dz;
                        sb[q] += dz * xv[q];
                    }
                }
        }
    }
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
        sh[0][threadIdx.x * VEC + q] = sa[q];
        sh[1][threadIdx.x * VEC + q] = sb[q];
    }
    __syncthreads();
    const int width = P.tx * VEC, c0 = (blockIdx.x % P.col_blocks) * width;
    for (int i = threadIdx.x; i < width && c0 + i < P.C; i += kGnThreads) {
        float s = 0.f, t = 0.f;
        for (int r = 0; r < P.ty; ++r) {
            s += sh[0][r * width + i];
            t += sh[1][r * width + i];
        }
        float *out = P.part + (static_cast<int64_t>(at.n) * P.slabs + at.slab) * 2 * P.C + c0 + i;
        out[0] = s;
        out[P.C] = t;
    }
}

// Blocks below `group_blocks`: one warp per image and group, S1 / (D HW) and
// S2 / (D HW).  The others: 32 channels each, 4 warps over the images' and
// slabs' partial sums, joined in a fixed order.
static __global__ void __launch_bounds__(128) gn_bwd_finish_kernel(const __grid_constant__ GnParams P,
                                                                   int32_t group_blocks) {
    __shared__ double sh[4][2][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (blockIdx.x < static_cast<unsigned>(group_blocks)) {
        const int64_t w = blockIdx.x * 4ll + warp;
        if (w >= static_cast<int64_t>(P.N) * P.G) return;
        const int n = static_cast<int>(w / P.G), g = static_cast<int>(w % P.G);
        const float *part = P.part + static_cast<int64_t>(n) * P.slabs * 2 * P.C + g * P.D;
        const int64_t entries = static_cast<int64_t>(P.slabs) * P.D;
        double s1 = 0.0, s2 = 0.0;
        for (int64_t e = lane; e < entries; e += 32) {
            const int64_t s = e / P.D;
            const int c = static_cast<int>(e % P.D);
            const double gamma = P.gamma ? P.gamma[g * P.D + c] : 1.f;
            s1 += gamma * part[s * 2 * P.C + c];
            s2 += gamma * part[(s * 2 + 1) * P.C + c];
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (lane == 0) {
            const double total = static_cast<double>(P.HW) * P.D;
            P.coef[w * 2] = static_cast<float>(s1 / total);
            P.coef[w * 2 + 1] = static_cast<float>(s2 / total);
        }
        return;
    }
    const int c = (blockIdx.x - group_blocks) * 32 + lane;
    double a = 0.0, b = 0.0;
    if (c < P.C)
        for (int64_t e = warp; e < static_cast<int64_t>(P.N) * P.slabs; e += 4) {
            a += P.part[e * 2 * P.C + c];
            b += P.part[(e * 2 + 1) * P.C + c];
        }
    sh[warp][0][lane] = a;
    sh[warp][1][lane] = b;
    __syncthreads();
    if (warp == 0 && c < P.C) {
        if (P.gbeta) P.gbeta[c] = static_cast<float>((sh[0][0][lane] + sh[1][0][lane]) + (sh[2][0][lane] + sh[3][0][lane]));
        if (P.ggamma) P.ggamma[c] = static_cast<float>((sh[0][1][lane] + sh[1][1][lane]) + (sh[2][1][lane] + sh[3][1][lane]));
    }
}

// gx = rstd (gamma dz - k1 - xhat k2).
template <typename T, int VEC>
__global__ void __launch_bounds__(kGnThreads) gn_bwd_apply_kernel(const __grid_constant__ GnParams P) {
    const GnPlace<VEC> at(P);
    if (!at.on) return;
    float mean[VEC], rstd[VEC], gamma[VEC], beta[VEC], k1[VEC], k2[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
        const int64_t s = static_cast<int64_t>(at.n) * P.G + (at.c + q) / P.D;
        mean[q] = P.mean[s];
        rstd[q] = P.rstd[s];
        gamma[q] = P.gamma ? P.gamma[at.c + q] : 1.f;
        beta[q] = P.beta ? P.beta[at.c + q] : 0.f;
        k1[q] = P.coef[s * 2];
        k2[q] = P.coef[s * 2 + 1];
    }
    const T *x = static_cast<const T *>(P.x.p) + at.n * P.x.sn + at.c;
    const T *g = static_cast<const T *>(P.g.p) + at.n * P.g.sn + at.c;
    T *o = static_cast<T *>(P.out) + at.n * P.on + at.c;
    constexpr int U = 2;
    for (int p = at.p0; p < at.p1; p += U * P.ty) {
        typename Pack<T, VEC>::Raw rx[U], rg[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (p + u * P.ty < at.p1) {
                rx[u] = Pack<T, VEC>::load(x + (p + static_cast<int64_t>(u) * P.ty) * P.x.sp);
                rg[u] = Pack<T, VEC>::load(g + (p + static_cast<int64_t>(u) * P.ty) * P.g.sp);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (p + u * P.ty < at.p1) {
                float xv[VEC], gv[VEC];
                Pack<T, VEC>::widen(rx[u], xv);
                Pack<T, VEC>::widen(rg[u], gv);
                float z[VEC], sl[VEC];
#pragma unroll
                for (int q = 0; q < VEC; ++q) {
                    xv[q] = (xv[q] - mean[q]) * rstd[q];
                    z[q] = xv[q] * gamma[q] + beta[q];
                }
                act_slopes(P.act, z, sl);
#pragma unroll
                for (int q = 0; q < VEC; ++q)
                    xv[q] = rstd[q] * (gamma[q] * gv[q] * sl[q] - k1[q] - xv[q] * k2[q]);
                Pack<T, VEC>::store(o + (p + static_cast<int64_t>(u) * P.ty) * P.op, xv);
            }
    }
}

// ---------------------------------------------------------------- one pass
__device__ __forceinline__ uint32_t gn_cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ float gn_ld_rank(const float *p, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void gn_cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void gn_cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <int BYTES>
__device__ __forceinline__ void gn_copy_async(void *dst, const void *src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}
template <int N>
__device__ __forceinline__ void gn_copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The tensor read once: a cluster of CTAs holds one image's chunk of whole
// groups on chip, each CTA a slab of its pixels.  A thread copies the vectors
// it will work on (fixed channels, every ty-th pixel) into its own slots of
// shared memory, all copies in flight at once, and reads them again for each
// pass; so no pass but the sums meets a barrier.  Sums go over the CTA's rows
// in shared memory and over the cluster through distributed shared memory,
// always in the same order.
template <typename T, int VEC>
struct GnChip {
    static constexpr int kBytes = VEC * sizeof(T);
    const GnParams &P;
    int n, chunk, rank, col, row, nt, cb, c, p0, count;
    bool on;
    T *xs, *gs;
    float *red, *part, *csum, *group;     // [nt][VEC], [256], [cb] x 2, [gpc] x 4

    __device__ __forceinline__ GnChip(const GnParams &p, uint8_t *smem, bool two) : P(p) {
        int b = blockIdx.x;
        rank = b % P.splits;
        b /= P.splits;
        chunk = b % P.chunks;
        n = b / P.chunks;
        col = threadIdx.x % P.tx;
        row = threadIdx.x / P.tx;
        nt = P.tx * P.ty;
        cb = P.tx * VEC;
        c = chunk * cb + col * VEC;
        on = row < P.ty;
        p0 = rank * P.slab + row;
        const int p1 = min(P.HW, (rank + 1) * P.slab);
        count = on && p0 < p1 ? (p1 - p0 + P.ty - 1) / P.ty : 0;
        xs = reinterpret_cast<T *>(smem) + threadIdx.x * VEC;
        uint8_t *end = smem + static_cast<size_t>(P.iters) * nt * kBytes;
        gs = nullptr;
        if (two) {
            gs = reinterpret_cast<T *>(end) + threadIdx.x * VEC;
            end += static_cast<size_t>(P.iters) * nt * kBytes;
        }
        red = reinterpret_cast<float *>(smem + (((end - smem) + 15) & ~static_cast<size_t>(15)));
        part = red + nt * VEC;
        csum = part + kGnThreads;
        group = csum + 2 * cb;
    }
    __device__ __forceinline__ const T *slot(const T *base, int i) const { return base + i * nt * VEC; }
    __device__ __forceinline__ T *slot(T *base, int i) const { return base + i * nt * VEC; }

    // Sums of v over the CTA's rows: csum[channel of the chunk].
    __device__ __forceinline__ void channel_sums(const float (&v)[VEC], float *out) {
        if (on)
#pragma unroll
            for (int q = 0; q < VEC; ++q) red[threadIdx.x * VEC + q] = v[q];
        __syncthreads();
        if (cb <= kGnThreads / 2) {
            const int parts = kGnThreads / cb, at = threadIdx.x / cb, ch = threadIdx.x - at * cb;
            float s = 0.f;
            if (at < parts)
                for (int r = at; r < P.ty; r += parts) s += red[r * cb + ch];
            part[threadIdx.x] = s;
            __syncthreads();
            if (threadIdx.x < cb) {
                s = 0.f;
                for (int k = 0; k < parts; ++k) s += part[k * cb + threadIdx.x];
                out[threadIdx.x] = s;
            }
        } else {
            for (int ch = threadIdx.x; ch < cb; ch += kGnThreads) {
                float s = 0.f;
                for (int r = 0; r < P.ty; ++r) s += red[r * cb + ch];
                out[ch] = s;
            }
        }
        __syncthreads();
    }
    // Sums of the channel sums over each group (times gamma), one warp a group.
    __device__ __forceinline__ void group_sums(const float *ch, const float *gamma, float *out) {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        for (int g = warp; g < P.gpc; g += kGnThreads / 32) {
            float s = 0.f;
            for (int d = lane; d < P.D; d += 32) {
                const int k = g * P.D + d;
                s += gamma ? gamma[chunk * cb + k] * ch[k] : ch[k];
            }
#pragma unroll
            for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            if (lane == 0) out[g] = s;
        }
    }
    // Everyone's `p` is written and may be read by the cluster.
    __device__ __forceinline__ void meet() {
        if (P.splits > 1) {
            gn_cluster_arrive();
            gn_cluster_wait();
        } else {
            __syncthreads();
        }
    }
    __device__ __forceinline__ float over_cluster(const float *p) const {
        if (P.splits == 1) return *p;
        float s = 0.f;
        for (int r = 0; r < P.splits; ++r) s += gn_ld_rank(p, r);
        return s;
    }
};

template <typename T, int VEC>
__global__ void __launch_bounds__(kGnThreads) gn_chip_fwd_kernel(const __grid_constant__ GnParams P) {
    extern __shared__ __align__(16) uint8_t gn_smem[];
    GnChip<T, VEC> K(P, gn_smem, false);
    const T *x = static_cast<const T *>(P.x.p) + K.n * P.x.sn + K.c;
    // four groups of copies, summed as they land
    const int quarter = (P.iters + 3) / 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int end = min(K.count, (k + 1) * quarter);
        for (int i = k * quarter; i < end; ++i)
            gn_copy_async<K.kBytes>(K.slot(K.xs, i), x + (K.p0 + static_cast<int64_t>(i) * P.ty) * P.x.sp);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    float acc[VEC] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (k == 0) gn_copy_wait<3>();
        if (k == 1) gn_copy_wait<2>();
        if (k == 2) gn_copy_wait<1>();
        if (k == 3) gn_copy_wait<0>();
        const int end = min(K.count, (k + 1) * quarter);
        for (int i = k * quarter; i < end; ++i) {
            float v[VEC];
            Pack<T, VEC>::widen(Pack<T, VEC>::load(K.slot(K.xs, i)), v);
#pragma unroll
            for (int q = 0; q < VEC; ++q) acc[q] += v[q];
        }
    }
    const float total = static_cast<float>(P.HW) * P.D;
    K.channel_sums(acc, K.csum);
    K.group_sums(K.csum, nullptr, K.group);
    K.meet();
    float *mean = K.group + 2 * P.gpc, *rstd = mean + P.gpc;
    for (int g = threadIdx.x; g < P.gpc; g += kGnThreads) mean[g] = K.over_cluster(K.group + g) / total;
    __syncthreads();
    float m[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
        m[q] = mean[(K.col * VEC + q) / P.D];
        acc[q] = 0.f;
    }
    for (int i = 0; i < K.count; ++i) {
        float v[VEC];
        Pack<T, VEC>::widen(Pack<T, VEC>::load(K.slot(K.xs, i)), v);
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
            const float d = v[q] - m[q];
            acc[q] = fmaf(d, d, acc[q]);
        }
    }
    K.channel_sums(acc, K.csum);
    K.group_sums(K.csum, nullptr, K.group + P.gpc);
    K.meet();
    for (int g = threadIdx.x; g < P.gpc; g += kGnThreads) {
        const float r = 1.f / sqrtf(K.over_cluster(K.group + P.gpc + g) / total + P.eps);
        rstd[g] = r;
        if (K.rank == 0) {
            const int64_t at = static_cast<int64_t>(K.n) * P.G + K.chunk * P.gpc + g;
            P.mean[at] = mean[g];
            P.rstd[at] = r;
        }
    }
    if (P.splits > 1) gn_cluster_arrive();   // the last remote read is done
    __syncthreads();
    float a[VEC], b[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
        a[q] = rstd[(K.col * VEC + q) / P.D] * (P.gamma && K.on ? P.gamma[K.c + q] : 1.f);
        b[q] = P.beta && K.on ? P.beta[K.c + q] : 0.f;
    }
    T *y = static_cast<T *>(P.out) + K.n * P.on + K.c;
    for (int i = 0; i < K.count; ++i) {
        float v[VEC];
        Pack<T, VEC>::widen(Pack<T, VEC>::load(K.slot(K.xs, i)), v);
#pragma unroll
        for (int q = 0; q < VEC; ++q) v[q] = (v[q] - m[q]) * a[q] + b[q];
        act_values(P.act, v);
        Pack<T, VEC>::store(y + (K.p0 + static_cast<int64_t>(i) * P.ty) * P.op, v);
    }
    if (P.splits > 1) gn_cluster_wait();
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kGnThreads) gn_chip_bwd_kernel(const __grid_constant__ GnParams P) {
    extern __shared__ __align__(16) uint8_t gn_smem[];
    GnChip<T, VEC> K(P, gn_smem, true);
    const T *x = static_cast<const T *>(P.x.p) + K.n * P.x.sn + K.c;
    const T *g = static_cast<const T *>(P.g.p) + K.n * P.g.sn + K.c;
    const int quarter = (P.iters + 3) / 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int end = min(K.count, (k + 1) * quarter);
        for (int i = k * quarter; i < end; ++i) {
            const int64_t p = K.p0 + static_cast<int64_t>(i) * P.ty;
            gn_copy_async<K.kBytes>(K.slot(K.xs, i), x + p * P.x.sp);
            gn_copy_async<K.kBytes>(K.slot(K.gs, i), g + p * P.g.sp);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    float mean[VEC], rstd[VEC], gamma[VEC], beta[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
        const int64_t at = static_cast<int64_t>(K.n) * P.G + (K.on ? (K.c + q) / P.D : 0);
        mean[q] = P.mean[at];
        rstd[q] = P.rstd[at];
        gamma[q] = P.gamma && K.on ? P.gamma[K.c + q] : 1.f;
        beta[q] = P.beta && K.on ? P.beta[K.c + q] : 0.f;
    }
    float sa[VEC] = {}, sb[VEC] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (k == 0) gn_copy_wait<3>();
        if (k == 1) gn_copy_wait<2>();
        if (k == 2) gn_copy_wait<1>();
        if (k == 3) gn_copy_wait<0>();
        const int end = min(K.count, (k + 1) * quarter);
        for (int i = k * quarter; i < end; ++i) {
            float xv[VEC], gv[VEC], z[VEC], sl[VEC];
            Pack<T, VEC>::widen(Pack<T, VEC>::load(K.slot(K.xs, i)), xv);
            Pack<T, VEC>::widen(Pack<T, VEC>::load(K.slot(K.gs, i)), gv);
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                xv[q] = (xv[q] - mean[q]) * rstd[q];
                z[q] = xv[q] * gamma[q] + beta[q];
            }
            act_slopes(P.act, z, sl);
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                gv[q] *= sl[q];
                sa[q] += gv[q];
                sb[q] += gv[q] * xv[q];
            }
            if constexpr (sizeof(T) == 4) {   // xhat and dz in the slots: not computed again
                Pack<T, VEC>::store(K.slot(K.xs, i), xv);
                Pack<T, VEC>::store(K.slot(K.gs, i), gv);
            }
        }
    }
    K.channel_sums(sa, K.csum);
    K.channel_sums(sb, K.csum + K.cb);
    K.group_sums(K.csum, P.gamma, K.group);
    K.group_sums(K.csum + K.cb, P.gamma, K.group + P.gpc);
    K.meet();
    const float total = static_cast<float>(P.HW) * P.D;
    float *k1 = K.group + 2 * P.gpc, *k2 = k1 + P.gpc;
    for (int j = threadIdx.x; j < P.gpc; j += kGnThreads) {
        k1[j] = K.over_cluster(K.group + j) / total;
        k2[j] = K.over_cluster(K.group + P.gpc + j) / total;
    }
    // the image's channel sums, for ggamma and gbeta: each CTA its share
    float *out = P.part + static_cast<int64_t>(K.n) * 2 * P.C + K.chunk * K.cb;
    for (int ch = threadIdx.x * P.splits + K.rank; ch < K.cb; ch += kGnThreads * P.splits) {
        out[ch] = K.over_cluster(K.csum + ch);
        out[P.C + ch] = K.over_cluster(K.csum + K.cb + ch);
    }
    if (P.splits > 1) gn_cluster_arrive();
    __syncthreads();
    float c1[VEC], c2[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
        c1[q] = k1[(K.col * VEC + q) / P.D];
        c2[q] = k2[(K.col * VEC + q) / P.D];
    }
    T *o = static_cast<T *>(P.out) + K.n * P.on + K.c;
    for (int i = 0; i < K.count; ++i) {
        float xv[VEC], gv[VEC];
        Pack<T, VEC>::widen(Pack<T, VEC>::load(K.slot(K.xs, i)), xv);
        Pack<T, VEC>::widen(Pack<T, VEC>::load(K.slot(K.gs, i)), gv);
        if constexpr (sizeof(T) != 4) {
            float z[VEC], sl[VEC];
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                xv[q] = (xv[q] - mean[q]) * rstd[q];
                z[q] = xv[q] * gamma[q] + beta[q];
            }
            act_slopes(P.act, z, sl);
#pragma unroll
            for (int q = 0; q < VEC; ++q) gv[q] *= sl[q];
        }
#pragma unroll
        for (int q = 0; q < VEC; ++q) gv[q] = rstd[q] * (gamma[q] * gv[q] - c1[q] - xv[q] * c2[q]);
        Pack<T, VEC>::store(o + (K.p0 + static_cast<int64_t>(i) * P.ty) * P.op, gv);
    }
    if (P.splits > 1) gn_cluster_wait();
}

}  // namespace mqc
