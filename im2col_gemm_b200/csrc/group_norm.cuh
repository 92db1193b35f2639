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
        if constexpr (sizeof(T) == 2 && VEC >= 2) {
            const uint32_t *w = reinterpret_cast<const uint32_t *>(&r);
#pragma unroll
            for (int q = 0; q < VEC / 2; ++q) {
                const float2 f = unpack2<T>(w[q]);
                v[2 * q] = f.x;
                v[2 * q + 1] = f.y;
            }
        } else {
            const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
            for (int q = 0; q < VEC; ++q) v[q] = to_f32(e[q]);
        }
    }
    __device__ static __forceinline__ void store(T *p, const float (&v)[VEC]) {
        Raw r;
        if constexpr (sizeof(T) == 2 && VEC >= 2) {
            uint32_t *w = reinterpret_cast<uint32_t *>(&r);
#pragma unroll
            for (int q = 0; q < VEC / 2; ++q) w[q] = pack2<T>(v[2 * q], v[2 * q + 1]);
        } else {
            T *e = reinterpret_cast<T *>(&r);
#pragma unroll
            for (int q = 0; q < VEC; ++q) e[q] = from_f32<T>(v[q]);
        }
        *reinterpret_cast<Raw *>(p) = r;
    }
};

// The group of each of VEC consecutive channels, from `c` on (D channels a
// group): one division, then counted on.  UNI: VEC divides D, one group.
template <int VEC, bool UNI, typename F>
__device__ __forceinline__ void per_channel_group(int c, int D, F &&f) {
    int g = c / D, left = D - (c - g * D);
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
        f(q, g);
        if (!UNI && --left == 0) {
            left = D;
            ++g;
        }
    }
}

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
    float *part;                         // backward: [N][slabs][2][C] sums of dz and dz xhat
    float *gpart;                        // two passes: [N][slabs][chunks * gpc][2] a group's (or piece's) sums
    float *ggamma, *gbeta;
    float eps;
    int32_t N, C, G, D, HW;
    int32_t act;
    // The split: channel chunks of gpc whole groups (or of 1 / pieces of one),
    // tx vectors wide; slabs of pixels, a thread taking every ty-th; `seg` sums
    // that a thread leaves for the groups of its vector (chip backward: threads
    // that share a channel's sum).
    int32_t chunks, gpc, pieces, width, tx, ty, slab, slabs, iters, threads, seg;
    int32_t splits;                      // on-chip form: CTAs of a cluster
    int32_t channel_blocks;              // backward, two passes: blocks that join the channels' sums
    FastDiv fd_tx, fd_ty, fd_chunks, fd_slabs, fd_cb, fd_entries;
};

constexpr int kGnThreads = 512;          // at most

__device__ __forceinline__ float warp_sum_f(float v, int from = 16) {
    for (int o = from; o > 0; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// VEC sums of a thread to shared memory, in wide stores: single words, VEC
// apart, would meet VEC-fold bank conflicts.
template <int VEC>
__device__ __forceinline__ void leave(float *at, const float (&v)[VEC]) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int q = 0; q < VEC; q += 4)
            *reinterpret_cast<float4 *>(at + q) = make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
    } else if constexpr (VEC == 2) {
        *reinterpret_cast<float2 *>(at) = make_float2(v[0], v[1]);
    } else {
        at[0] = v[0];
    }
}

// Sums over the CTA of f(channel of the thread's vector) by group, one warp a
// group, given to out(group of the chunk, sum) in lane 0.  A thread leaves
// seg values: one (UNI), VEC / D, or VEC; `per` of them belong to a group in
// a row.  red: tx * ty * seg floats.
template <int VEC, bool UNI, typename F, typename O>
__device__ __forceinline__ void group_reduce(const GnParams &P, float *red, bool on, F &&f, O &&out) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    const int seg = UNI ? 1 : P.seg;
    if (on) {
        if (UNI || seg != VEC) {
            const int len = VEC / seg;
            float s = 0.f;
            int at = threadIdx.x * seg, left = len;
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                s += f(q);
                if (UNI ? q == VEC - 1 : --left == 0) {
                    red[at++] = s;
                    s = 0.f;
                    left = len;
                }
            }
        } else {
            float v[VEC];
#pragma unroll
            for (int q = 0; q < VEC; ++q) v[q] = f(q);
            leave<VEC>(red + threadIdx.x * VEC, v);
        }
    }
    __syncthreads();
    const int per = P.fd_entries.d, total = per * P.ty, width = P.tx * seg;
    for (int g = warp; g < P.gpc; g += warps) {
        float s = 0.f;
        for (int e = lane; e < total; e += 32) {
            const int r = per == 1 ? e : P.fd_entries.div(e);
            s += red[r * width + g * per + (e - r * per)];
        }
        s = warp_sum_f(s);
        if (lane == 0) out(g, s);
    }
}

// A thread's running statistics of its channels, about its first value of
// each: that value being one of them, the difference of the squares loses at
// most a factor of their number (never one of mean^2 / variance).
template <int VEC>
struct GnRunning {
    float first[VEC], sum[VEC], sq[VEC];
    __device__ __forceinline__ GnRunning() {
#pragma unroll
        for (int q = 0; q < VEC; ++q) first[q] = sum[q] = sq[q] = 0.f;
    }
    __device__ __forceinline__ void start(const float (&v)[VEC]) {
#pragma unroll
        for (int q = 0; q < VEC; ++q) first[q] = isfinite(v[q]) ? -v[q] : 0.f;   // an infinite mean stays infinite
    }
    __device__ __forceinline__ void add(float (&v)[VEC]) {
        add_to(v, first);
        add_to(sum, v);
        fma_to(sq, v, v, sq);
    }
    // sum -> mean, sq -> squared deviations from it
    __device__ __forceinline__ void finish(int count) {
        const float inv = count > 0 ? 1.f / static_cast<float>(count) : 0.f;
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
            const float d = sum[q] * inv;
            sq[q] = fmaf(-sum[q], d, sq[q]);
            sum[q] = d - first[q];
        }
    }
};

// Channels' sums joined over `rows` partial rows ([row][2][C]), 32 channels a
// block, a warp every (blockDim / 32)-th row with eight loads in flight; the
// warps' shares in warp order.  sh: [warps][2][32] doubles.
__device__ __forceinline__ void join_channels(const GnParams &P, int block, int64_t rows, double *sh) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const int c = block * 32 + lane;
    double a = 0.0, b = 0.0;
    if (c < P.C) {
        const float *at = P.part + c;
        for (int64_t e = warp; e < rows; e += 8 * warps) {
            float va[8], vb[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int64_t r = e + u * warps;
                va[u] = r < rows ? at[r * 2 * P.C] : 0.f;
                vb[u] = r < rows ? at[(r * 2 + 1) * P.C] : 0.f;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                a += va[u];
                b += vb[u];
            }
        }
    }
    sh[(warp * 2) * 32 + lane] = a;
    sh[(warp * 2 + 1) * 32 + lane] = b;
    __syncthreads();
    if (warp < 2 && c < P.C) {   // warp 0: gbeta, warp 1: ggamma
        double s = 0.0;
        for (int k = 0; k < warps; ++k) s += sh[(k * 2 + warp) * 32 + lane];
        float *out = warp == 0 ? P.gbeta : P.ggamma;
        if (out) out[c] = static_cast<float>(s);
    }
}
static __global__ void __launch_bounds__(kGnThreads) gn_channels_kernel(const __grid_constant__ GnParams P,
                                                                        int64_t rows) {
    __shared__ double sh[kGnThreads / 32 * 2 * 32];
    wait_previous();
    join_channels(P, blockIdx.x, rows, sh);
}

// Backward: the CTA's sums of dz (sa) and dz xhat (sb) by channel: csum[cb] and
// csum[cb ..].  In two steps when there are threads to share a channel.  red:
// 2 tx ty VEC floats, part: 2 blockDim, parts: threads that share a channel.
template <int VEC>
__device__ __forceinline__ void channel_sums(const GnParams &P, float *red, float *part, float *csum, bool on,
                                             const float (&sa)[VEC], const float (&sb)[VEC]) {
    const int threads = blockDim.x, nt = P.tx * P.ty, cb = P.tx * VEC;
    float *redb = red + nt * VEC;
    if (on) {
        leave<VEC>(red + threadIdx.x * VEC, sa);
        leave<VEC>(redb + threadIdx.x * VEC, sb);
    }
    __syncthreads();
    if (cb <= threads / 2) {
        const int parts = P.seg, at = P.fd_cb.div(threadIdx.x), ch = threadIdx.x - at * cb;
        float s = 0.f, t = 0.f;
        if (at < parts)
            for (int r = at; r < P.ty; r += parts) {
                s += red[r * cb + ch];
                t += redb[r * cb + ch];
            }
        part[threadIdx.x] = s;
        part[threads + threadIdx.x] = t;
        __syncthreads();
        for (int j = threadIdx.x; j < 2 * cb; j += threads) {
            const int from = j >= cb ? threads + j - cb : j;
            float v = 0.f;
            for (int k = 0; k < parts; ++k) v += part[from + k * cb];
            csum[j] = v;
        }
    } else {
        for (int ch = threadIdx.x; ch < cb; ch += threads) {
            float s = 0.f, t = 0.f;
            for (int r = 0; r < P.ty; ++r) {
                s += red[r * cb + ch];
                t += redb[r * cb + ch];
            }
            csum[ch] = s;
            csum[cb + ch] = t;
        }
    }
    __syncthreads();
}
// Their sums times gamma over the `channels` of each of the chunk's groups,
// one warp a group.  c0: the chunk's first channel.
template <typename O>
__device__ __forceinline__ void gamma_sums(const GnParams &P, const float *csum, int cb, int c0, int channels, O &&out) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    for (int g = warp; g < P.gpc; g += warps) {
        float s = 0.f, t = 0.f;
        for (int d = lane; d < channels; d += 32) {
            const int k = g * P.D + d;
            const float ga = P.gamma ? P.gamma[c0 + k] : 1.f;
            s = fmaf(ga, csum[k], s);
            t = fmaf(ga, csum[cb + k], t);
        }
        s = warp_sum_f(s);
        t = warp_sum_f(t);
        if (lane == 0) out(g, s, t);
    }
}

// ---------------------------------------------------------------- two passes
constexpr int kPassThreads = 256;

// The block's image, slab and chunk, and this thread's place in it.
template <int VEC>
struct GnPlace {
    int n, slab, chunk, row, col, c, p0, pixels, count, c_end;
    bool on;
    __device__ __forceinline__ GnPlace(const GnParams &P, int block) {
        int b = P.fd_chunks.div(block);
        chunk = block - b * P.chunks;
        n = P.fd_slabs.div(b);
        slab = b - n * P.slabs;
        row = P.fd_tx.div(threadIdx.x);
        col = threadIdx.x - row * P.tx;
        // a piece of a group ends with the group
        const int group = P.pieces > 1 ? chunk / P.pieces : chunk;
        const int c0 = P.pieces > 1 ? group * P.D + (chunk - group * P.pieces) * P.width : chunk * P.width;
        c_end = P.pieces > 1 ? min(c0 + P.width, (group + 1) * P.D) : c0 + P.width;
        c = c0 + col * VEC;
        on = row < P.ty && c < c_end;
        const int first = slab * P.slab;
        pixels = min(P.HW - first, P.slab);
        p0 = first + row;
        count = on && row < pixels ? P.fd_ty.div(pixels - row - 1) + 1 : 0;
    }
    // Channels of a group in this chunk, and the group's number in the image.
    __device__ __forceinline__ int channels(const GnParams &P) const {
        return P.pieces > 1 ? min(P.width, P.D - (chunk % P.pieces) * P.width) : P.D;
    }
    __device__ __forceinline__ int group(const GnParams &P, int g) const {
        return P.pieces > 1 ? chunk / P.pieces : chunk * P.gpc + g;
    }
};

template <int BYTES>
__device__ __forceinline__ void gn_copy_async(uint32_t dst, const void *src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
template <int N>
__device__ __forceinline__ void gn_copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A thread's reads of its vectors of NT tensors, kRing of them under way: they
// land in its own slots of shared memory ([slot][tensor][thread]), so the depth
// costs no registers and the order needs no barrier.  (Batches loaded ahead
// into registers: 16x64x160x160 bf16 forward took 38.9 us, now 34.7, and
// 32x128x80x80 fp32 backward 100.6, now 88.7.)  Elements of two
// bytes, too small for asynchronous copies, are loaded when they are due.
template <typename T, int VEC, int NT>
struct GnRing {
    static constexpr int kBytes = VEC * sizeof(T);
    static constexpr int kRing = kBytes * NT <= 16 ? 8 : 4;
    static constexpr bool kAsync = kBytes >= 4;
    using V = Pack<T, VEC>;
    const T *due[NT], *ahead[NT];        // the next vector to be taken, to be asked for
    int64_t step[NT];
    uint8_t *slots;
    int count;

    static constexpr int kSlotBytes = kAsync ? kRing * NT * kPassThreads * kBytes : 0;
    __device__ __forceinline__ GnRing(uint8_t *smem, int n) : slots(smem + threadIdx.x * kBytes), count(n) {}
    __device__ __forceinline__ void ask(int i) {
        if (!kAsync) return;
        if (i < count) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                gn_copy_async<kBytes < 4 ? 4 : kBytes>(
                    smem_u32(slots + ((i & (kRing - 1)) * NT + t) * kPassThreads * kBytes), ahead[t]);
                ahead[t] += step[t];
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void begin() {
#pragma unroll
        for (int t = 0; t < NT; ++t) ahead[t] = due[t];
#pragma unroll
        for (int i = 0; i < kRing; ++i) ask(i);
    }
    // The i-th vectors, and the request for those that take their place.
    __device__ __forceinline__ void take(int i, typename V::Raw (&r)[NT]) {
        if (kAsync) gn_copy_wait<kRing - 1>();
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (kAsync) {
                r[t] = V::load(reinterpret_cast<const T *>(slots + ((i & (kRing - 1)) * NT + t) * kPassThreads * kBytes));
            } else {
                r[t] = V::load(due[t]);
                due[t] += step[t];
            }
        }
        ask(i + kRing);
    }
};

// First pass: mean and squared deviations of each group (or piece) of the slab,
// about the thread's first value, joined by means and squared deviations (Chan
// et al.): no large squares are subtracted.  Both forward passes together read
// 16x64x160x160 bf16 twice and write it once (157 MB) in 32.3 us, 4.9 TB/s;
// read once it would take 16.3, but a group (four channels, 205 KB) does not
// quite fit an SM in rows of 8 bytes, and the chunk of 32 channels (1.6 MB, rows
// of 64 bytes) that the on-chip plan prefers took clusters of 16 and 44 us.
// (Four groups, 819 KB in rows of 32 bytes, were not timed.)
template <typename T, int VEC, bool UNI>
__global__ void __launch_bounds__(kPassThreads, 3) gn_stats_kernel(const __grid_constant__ GnParams P) {
    extern __shared__ __align__(16) uint8_t gn_smem[];
    let_next_start();
    using V = Pack<T, VEC>;
    const GnPlace<VEC> at(P, blockIdx.x);
    using Ring = GnRing<T, VEC, 1>;
    Ring ring(gn_smem, at.count);
    ring.due[0] = static_cast<const T *>(P.x.p) + at.n * P.x.sn + at.c + at.p0 * P.x.sp;
    ring.step[0] = P.ty * P.x.sp;
    ring.begin();
    GnRunning<VEC> run;
#pragma unroll 4
    for (int i = 0; i < at.count; ++i) {
        typename V::Raw r[1];
        ring.take(i, r);
        float v[VEC];
        V::widen(r[0], v);
        if (i == 0) run.start(v);
        run.add(v);
    }
    __syncthreads();   // the sums take the slots' place
    float *gn_red = reinterpret_cast<float *>(gn_smem);
    run.finish(at.count);
    const int nt = P.tx * P.ty, seg = UNI ? 1 : P.seg;
    float *mean = gn_red + nt * seg;
    const float cnt = static_cast<float>(at.count);
    const float total = static_cast<float>(at.pixels) * at.channels(P);
    float2 *out = reinterpret_cast<float2 *>(P.gpart) +
                  ((static_cast<int64_t>(at.n) * P.slabs + at.slab) * P.chunks + at.chunk) * P.gpc;
    group_reduce<VEC, UNI>(P, gn_red, at.row < P.ty, [&](int q) { return cnt * run.sum[q]; },
                           [&](int g, float s) { mean[g] = s / total; });
    __syncthreads();
    float m[VEC];
    per_channel_group<VEC, UNI>(at.col * VEC, P.D, [&](int q, int g) { m[q] = mean[g]; });
    group_reduce<VEC, UNI>(P, gn_red, at.row < P.ty,
                           [&](int q) { return fmaf(cnt * (run.sum[q] - m[q]), run.sum[q] - m[q], run.sq[q]); },
                           [&](int g, float s) { out[g] = make_float2(mean[g], s); });
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sums over the partial results (pairs) of each group of the block's chunk, all
// slabs and pieces: f(first pair, pair, the values it covers, sums) adds one to
// a pair of sums, out(group, first pair, sums) gets the total.  Neighbouring
// threads read neighbouring groups, and each has four loads under way: with two
// images the pairs of some 200 slabs are read by every block (a warp a group,
// one load after another, 2x128x80x80 fp32 took 20.6 us, now 11.8).
constexpr int kJoinBytes = kPassThreads * sizeof(double2);
template <int VEC, typename F, typename O>
__device__ __forceinline__ void join_parts(const GnParams &P, const GnPlace<VEC> &at, double2 *sh, F &&f, O &&out) {
    const float2 *part = reinterpret_cast<const float2 *>(P.gpart) + static_cast<int64_t>(at.n) * P.slabs * P.chunks * P.gpc;
    const int first = P.pieces > 1 ? at.chunk - at.chunk % P.pieces : at.chunk, rows = P.slabs * P.pieces;
    const int per = kPassThreads / P.gpc;   // a chunk of whole groups has 256 of them at most
    const int r = threadIdx.x / P.gpc, g = threadIdx.x - r * P.gpc;
    const float2 *from = part + static_cast<int64_t>(first) * P.gpc;
    if (r < per) {
        const float2 head = from[g];
        double2 sum = make_double2(0.0, 0.0);
        for (int e0 = r; e0 < rows; e0 += 4 * per) {
            float2 v[4];
            float n[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int e = e0 + u * per;
                const int s = P.pieces > 1 ? e / P.pieces : e, k = e - s * P.pieces;
                const int channels = P.pieces > 1 ? min(P.width, P.D - k * P.width) : P.D;
                n[u] = static_cast<float>(min(P.HW - s * P.slab, P.slab)) * channels;
                if (e < rows) v[u] = from[(static_cast<int64_t>(s) * P.chunks + k) * P.gpc + g];
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (e0 + u * per < rows) f(head, v[u], n[u], sum);
        }
        sh[threadIdx.x] = sum;
    }
    __syncthreads();
    if (per <= 16) {
        if (r == 0) {
            double2 sum = sh[g];
            for (int k = 1; k < per; ++k) {
                sum.x += sh[k * P.gpc + g].x;
                sum.y += sh[k * P.gpc + g].y;
            }
            out(g, from[g], sum);
        }
    } else {
        for (int j = threadIdx.x / 32; j < P.gpc; j += kPassThreads / 32) {
            double2 sum = make_double2(0.0, 0.0);
            for (int k = threadIdx.x % 32; k < per; k += 32) {
                sum.x += sh[k * P.gpc + j].x;
                sum.y += sh[k * P.gpc + j].y;
            }
            sum.x = warp_sum(sum.x);
            sum.y = warp_sum(sum.y);
            if (threadIdx.x % 32 == 0) out(j, from[j], sum);
        }
    }
    __syncthreads();
}

// Second pass: y = act((x - mean) (rstd gamma) + beta).  Blocks go from the
// last image to the first, so that what the first pass read last is still in
// L2.  The first loads are under way while the statistics are joined.
template <typename T, int VEC, bool UNI>
__global__ void __launch_bounds__(kPassThreads, 3) gn_apply_kernel(const __grid_constant__ GnParams P) {
    extern __shared__ __align__(16) uint8_t gn_smem[];
    using V = Pack<T, VEC>;
    using Ring = GnRing<T, VEC, 1>;
    const GnPlace<VEC> at(P, gridDim.x - 1 - blockIdx.x);
    float *mean = reinterpret_cast<float *>(gn_smem + Ring::kSlotBytes + kJoinBytes), *rstd = mean + P.gpc;
    Ring ring(gn_smem, at.count);
    ring.due[0] = static_cast<const T *>(P.x.p) + at.n * P.x.sn + at.c + at.p0 * P.x.sp;
    ring.step[0] = P.ty * P.x.sp;
    ring.begin();
    T *y = static_cast<T *>(P.out) + at.n * P.on + at.c + at.p0 * P.op;
    const int64_t ystep = P.ty * P.op;
    float a[VEC], b[VEC], m[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
        a[q] = P.gamma && at.on ? P.gamma[at.c + q] : 1.f;
        b[q] = P.beta && at.on ? P.beta[at.c + q] : 0.f;
    }
    wait_previous();
    // Means about the first slab's (0 if that is not finite), in 64 bits: what
    // cancels in the deviations is the spread of the slabs' means alone.
    const double total = static_cast<double>(P.HW) * P.D;
    join_parts(P, at, reinterpret_cast<double2 *>(gn_smem + Ring::kSlotBytes),
               [](float2 head, float2 v, float n, double2 &sum) {
                   const double d = static_cast<double>(v.x) - (isfinite(head.x) ? head.x : 0.f);
                   sum.x += n * d;
                   sum.y += v.y + n * d * d;
               },
               [&](int g, float2 head, double2 sum) {
                   const double d = sum.x / total, var = fmax(sum.y / total - d * d, 0.0);
                   mean[g] = static_cast<float>((isfinite(head.x) ? head.x : 0.f) + d);
                   rstd[g] = static_cast<float>(1.0 / sqrt((isfinite(d) ? var : d - d) + P.eps));
                   if (at.slab == 0 && (P.pieces == 1 || at.chunk % P.pieces == 0)) {
                       const int64_t i = static_cast<int64_t>(at.n) * P.G + at.group(P, g);
                       P.mean[i] = mean[g];
                       P.rstd[i] = rstd[g];
                   }
               });
    per_channel_group<VEC, UNI>(at.col * VEC, P.D, [&](int q, int g) {
        m[q] = -mean[g];
        a[q] *= rstd[g];
    });
#pragma unroll 2
    for (int i = 0; i < at.count; ++i, y += ystep) {
        typename V::Raw r[1];
        ring.take(i, r);
        float v[VEC];
        V::widen(r[0], v);
        add_to(v, m);
        fma_to(v, v, a, b);
        act_values<true>(P.act, v);
        V::store(y, v);
    }
}

// What the backward pass keeps of a thread's channels.
template <int VEC>
struct GnSlope {
    float mean[VEC], rstd[VEC], gamma[VEC], beta[VEC];
    template <bool UNI>
    __device__ __forceinline__ void load(const GnParams &P, int n, int group0, int inner, int c, bool on) {
        per_channel_group<VEC, UNI>(on ? inner : 0, P.D, [&](int q, int g) {
            const int64_t at = static_cast<int64_t>(n) * P.G + group0 + (on ? g : 0);
            mean[q] = -P.mean[at];
            rstd[q] = P.rstd[at];
            gamma[q] = P.gamma && on ? P.gamma[c + q] : 1.f;
            beta[q] = P.beta && on ? P.beta[c + q] : 0.f;
        });
    }
    // x -> xhat, g -> dz
    __device__ __forceinline__ void apply(int act, float (&x)[VEC], float (&g)[VEC]) const {
        float z[VEC], sl[VEC];
        add_to(x, mean);
        mul_to(x, rstd);
        fma_to(z, x, gamma, beta);
        act_slopes<true>(act, z, sl);
        mul_to(g, sl);
    }
};

// First pass: sums of dz and dz xhat, by channel and (times gamma) by group.
// dz is computed again by the second pass: both passes read x and g (and SiLU's
// exponential, twice, keeps the issue slots half busy).  32x128x80x80 fp32:
// 524 MB in 84 us, 6.2 TB/s; 128x256x14x14 bf16 (64 MB) 19.6 us.
template <typename T, int VEC, bool UNI>
__global__ void __launch_bounds__(kPassThreads, 3) gn_bwd_sums_kernel(const __grid_constant__ GnParams P) {
    extern __shared__ __align__(16) uint8_t gn_smem[];
    let_next_start();
    using V = Pack<T, VEC>;
    using Ring = GnRing<T, VEC, 2>;
    const GnPlace<VEC> at(P, blockIdx.x);
    Ring ring(gn_smem, at.count);
    ring.due[0] = static_cast<const T *>(P.x.p) + at.n * P.x.sn + at.c + at.p0 * P.x.sp;
    ring.due[1] = static_cast<const T *>(P.g.p) + at.n * P.g.sn + at.c + at.p0 * P.g.sp;
    ring.step[0] = P.ty * P.x.sp;
    ring.step[1] = P.ty * P.g.sp;
    ring.begin();
    GnSlope<VEC> K;
    K.template load<UNI>(P, at.n, at.group(P, 0), at.col * VEC, at.c, at.on);
    float sa[VEC] = {}, sb[VEC] = {};
#pragma unroll 2
    for (int i = 0; i < at.count; ++i) {
        typename V::Raw r[2];
        ring.take(i, r);
        float xv[VEC], gv[VEC];
        V::widen(r[0], xv);
        V::widen(r[1], gv);
        K.apply(P.act, xv, gv);
        add_to(sa, gv);
        fma_to(sb, gv, xv, sb);
    }
    __syncthreads();   // the sums take the slots' place
    float *gn_red = reinterpret_cast<float *>(gn_smem);
    const int nt = P.tx * P.ty, cb = P.tx * VEC, c0 = at.c - at.col * VEC;
    float *part = gn_red + 2 * nt * VEC, *csum = part + 2 * blockDim.x;
    channel_sums<VEC>(P, gn_red, part, csum, at.row < P.ty, sa, sb);
    float *out = P.part + (static_cast<int64_t>(at.n) * P.slabs + at.slab) * 2 * P.C + c0;
    for (int ch = threadIdx.x; ch < at.c_end - c0; ch += blockDim.x) {
        out[ch] = csum[ch];
        out[P.C + ch] = csum[cb + ch];
    }
    float2 *gout = reinterpret_cast<float2 *>(P.gpart) +
                   ((static_cast<int64_t>(at.n) * P.slabs + at.slab) * P.chunks + at.chunk) * P.gpc;
    gamma_sums(P, csum, cb, c0, at.channels(P), [&](int g, float s, float t) { gout[g] = make_float2(s, t); });
}

// Second pass: gx = rstd gamma dz - (rstd k1 + xhat rstd k2), from the last
// image to the first.  The first channel_blocks blocks join the channels' sums
// instead.
template <typename T, int VEC, bool UNI>
__global__ void __launch_bounds__(kPassThreads, 3) gn_bwd_apply_kernel(const __grid_constant__ GnParams P) {
    extern __shared__ __align__(16) uint8_t gn_smem[];
    using V = Pack<T, VEC>;
    using Ring = GnRing<T, VEC, 2>;
    if (blockIdx.x < P.channel_blocks) {
        wait_previous();
        join_channels(P, blockIdx.x, static_cast<int64_t>(P.N) * P.slabs, reinterpret_cast<double *>(gn_smem));
        return;
    }
    const GnPlace<VEC> at(P, gridDim.x - 1 - blockIdx.x);
    const int group0 = at.group(P, 0);
    float *k1 = reinterpret_cast<float *>(gn_smem + Ring::kSlotBytes + kJoinBytes), *k2 = k1 + P.gpc;
    Ring ring(gn_smem, at.count);
    ring.due[0] = static_cast<const T *>(P.x.p) + at.n * P.x.sn + at.c + at.p0 * P.x.sp;
    ring.due[1] = static_cast<const T *>(P.g.p) + at.n * P.g.sn + at.c + at.p0 * P.g.sp;
    ring.step[0] = P.ty * P.x.sp;
    ring.step[1] = P.ty * P.g.sp;
    ring.begin();
    T *o = static_cast<T *>(P.out) + at.n * P.on + at.c + at.p0 * P.op;
    const int64_t ostep = P.ty * P.op;
    GnSlope<VEC> K;
    K.template load<UNI>(P, at.n, group0, at.col * VEC, at.c, at.on);
    wait_previous();
    const double total = static_cast<double>(P.HW) * P.D;
    join_parts(P, at, reinterpret_cast<double2 *>(gn_smem + Ring::kSlotBytes),
               [](float2, float2 v, float, double2 &sum) {
                   sum.x += v.x;
                   sum.y += v.y;
               },
               [&](int j, float2, double2 sum) {
                   k1[j] = static_cast<float>(sum.x / total);
                   k2[j] = static_cast<float>(sum.y / total);
               });
    float scale[VEC], c1[VEC], c2[VEC];
    per_channel_group<VEC, UNI>(at.col * VEC, P.D, [&](int q, int j) {
        scale[q] = K.rstd[q] * K.gamma[q];
        c1[q] = -K.rstd[q] * k1[j];
        c2[q] = -K.rstd[q] * k2[j];
    });
#pragma unroll 2
    for (int i = 0; i < at.count; ++i, o += ostep) {
        typename V::Raw r[2];
        ring.take(i, r);
        float xv[VEC], gv[VEC];
        V::widen(r[0], xv);
        V::widen(r[1], gv);
        K.apply(P.act, xv, gv);
        fma_to(xv, xv, c2, c1);
        fma_to(gv, gv, scale, xv);
        V::store(o, gv);
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
// (The lanes of a warp come from loops and branches of their own.)
__device__ __forceinline__ void gn_cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void gn_cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t gn_cluster_id() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
    return r;
}

// The tensor read once: a cluster of CTAs holds one image's chunk of whole
// groups on chip, each CTA a slab of its pixels.  A thread copies the vectors
// it will work on (fixed channels, every ty-th pixel) into its own slots of
// shared memory, all copies in flight at once, and reads them again for the
// second pass; so only the sums meet barriers.  Sums go over the CTA in shared
// memory and over the cluster through distributed shared memory, always in the
// same order.  Bound by latency (the copies, two barriers, the stores, one
// after another) unless several CTAs share an SM: 1x256x14x14 bf16 4.4 us;
// 7x320x45x37 fp32 (30 MB, 112 CTAs of 147 KB, not quite one an SM) 11.9.
template <typename T, int VEC>
struct GnChip {
    static constexpr int kBytes = VEC * sizeof(T);
    const GnParams &P;
    int n, chunk, rank, col, row, nt, cb, c, p0, count, pixels;
    bool on;
    T *xs, *gs;
    float *red;                          // row sums

    __device__ __forceinline__ GnChip(const GnParams &p, uint8_t *smem, bool two) : P(p) {
        const int id = gn_cluster_id();
        rank = gn_cluster_rank();
        n = P.fd_chunks.div(id);
        chunk = id - n * P.chunks;
        row = P.fd_tx.div(threadIdx.x);
        col = threadIdx.x - row * P.tx;
        nt = P.tx * P.ty;
        cb = P.tx * VEC;
        c = chunk * cb + col * VEC;
        on = row < P.ty;
        const int first = rank * P.slab;
        pixels = min(P.HW - first, P.slab);
        p0 = first + row;
        count = on && row < pixels ? P.fd_ty.div(pixels - row - 1) + 1 : 0;
        xs = reinterpret_cast<T *>(smem) + threadIdx.x * VEC;
        const int bytes = P.iters * nt * kBytes;
        gs = reinterpret_cast<T *>(smem + bytes) + threadIdx.x * VEC;
        red = reinterpret_cast<float *>(smem + ((bytes * (two ? 2 : 1) + 15) & ~15));
    }
    __device__ __forceinline__ int quarter(int k) const { return min(count, (k * P.iters + 3) / 4); }
    // Everyone's sums are written and may be read by the cluster.
    __device__ __forceinline__ void meet() const {
        if (P.splits > 1) {
            gn_cluster_arrive();
            gn_cluster_wait();
        } else {
            __syncthreads();
        }
    }
};

// The CTA joins its threads, and the cluster its CTAs, by means and squared
// deviations (Chan et al.).
template <typename T, int VEC, bool UNI>
__global__ void __launch_bounds__(kGnThreads) gn_chip_fwd_kernel(const __grid_constant__ GnParams P) {
    extern __shared__ __align__(16) uint8_t gn_smem[];
    using V = Pack<T, VEC>;
    GnChip<T, VEC> K(P, gn_smem, false);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    const int seg = UNI ? 1 : P.seg;
    float *sums = K.red + K.nt * seg;            // [gpc] x 4: CTA's means, squares; mean, rstd
    float *dev = sums + P.gpc, *mean = dev + P.gpc, *rstd = mean + P.gpc;
    const int stride = K.nt * VEC;               // between a thread's slots
    {
        const T *x = static_cast<const T *>(P.x.p) + K.n * P.x.sn + K.c + K.p0 * P.x.sp;
        const int64_t step = P.ty * P.x.sp;
        uint32_t dst = smem_u32(K.xs);
        // four groups of copies, summed as they land
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int end = K.quarter(k + 1);
            for (int i = K.quarter(k); i < end; ++i) {
                gn_copy_async<K.kBytes>(dst, x);
                x += step;
                dst += stride * sizeof(T);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }
    float a[VEC], b[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
        a[q] = P.gamma && K.on ? P.gamma[K.c + q] : 1.f;
        b[q] = P.beta && K.on ? P.beta[K.c + q] : 0.f;
    }
    GnRunning<VEC> run;
    const T *slot = K.xs;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (k == 0) gn_copy_wait<3>();
        if (k == 1) gn_copy_wait<2>();
        if (k == 2) gn_copy_wait<1>();
        if (k == 3) gn_copy_wait<0>();
        if (k == 0 && K.count > 0) {
            float v[VEC];
            V::widen(V::load(slot), v);
            run.start(v);
        }
        const int end = K.quarter(k + 1);
#pragma unroll 2
        for (int i = K.quarter(k); i < end; ++i, slot += stride) {
            float v[VEC];
            V::widen(V::load(slot), v);
            run.add(v);
        }
    }
    run.finish(K.count);
    const float cnt = static_cast<float>(K.count);
    const float here = static_cast<float>(K.pixels) * P.D;
    group_reduce<VEC, UNI>(P, K.red, K.on, [&](int q) { return cnt * run.sum[q]; },
                           [&](int g, float s) { sums[g] = s / here; });
    __syncthreads();
    float m[VEC];
    per_channel_group<VEC, UNI>(K.col * VEC, P.D, [&](int q, int g) { m[q] = sums[g]; });
    group_reduce<VEC, UNI>(P, K.red, K.on,
                           [&](int q) { return fmaf(cnt * (run.sum[q] - m[q]), run.sum[q] - m[q], run.sq[q]); },
                           [&](int g, float s) { dev[g] = s; });
    K.meet();
    const float total = static_cast<float>(P.HW) * P.D;
    for (int g = warp; g < P.gpc; g += warps) {
        float mu = sums[g], s2 = dev[g];
        if (P.splits > 1) {   // one lane a CTA
            const bool in = lane < P.splits;
            const float n = in ? static_cast<float>(min(P.HW - lane * P.slab, P.slab)) * P.D : 0.f;
            const float mr = in ? gn_ld_rank(sums + g, lane) : 0.f, sr = in ? gn_ld_rank(dev + g, lane) : 0.f;
            // about the first CTA's mean (0 if that is not finite), so that equal means stay exact
            const float head = __shfl_sync(0xFFFFFFFFu, mr, 0), base = isfinite(head) ? head : 0.f;
            mu = base + warp_sum_f(in ? n * (mr - base) : 0.f, 8) / total;
            mu = __shfl_sync(0xFFFFFFFFu, mu, 0);
            s2 = warp_sum_f(in ? fmaf(n * (mr - mu), mr - mu, sr) : 0.f, 8);
        }
        if (lane == 0) {
            const float r = 1.f / sqrtf(s2 / total + P.eps);
            mean[g] = mu;
            rstd[g] = r;
            if (K.rank == 0) {
                const int64_t at = static_cast<int64_t>(K.n) * P.G + K.chunk * P.gpc + g;
                P.mean[at] = mu;
                P.rstd[at] = r;
            }
        }
    }
    if (P.splits > 1) gn_cluster_arrive();   // the last remote read is done
    __syncthreads();
    per_channel_group<VEC, UNI>(K.col * VEC, P.D, [&](int q, int g) {
        m[q] = -mean[g];
        a[q] *= rstd[g];
    });
    T *y = static_cast<T *>(P.out) + K.n * P.on + K.c + K.p0 * P.op;
    const int64_t step = P.ty * P.op;
    slot = K.xs;
#pragma unroll 2
    for (int i = 0; i < K.count; ++i, slot += stride, y += step) {
        float v[VEC];
        V::widen(V::load(slot), v);
        add_to(v, m);
        fma_to(v, v, a, b);
        act_values<true>(P.act, v);
        V::store(y, v);
    }
    if (P.splits > 1) gn_cluster_wait();
}

// Backward.
template <typename T, int VEC, bool UNI>
__global__ void __launch_bounds__(kGnThreads) gn_chip_bwd_kernel(const __grid_constant__ GnParams P) {
    let_next_start();   // gn_channels_kernel
    extern __shared__ __align__(16) uint8_t gn_smem[];
    using V = Pack<T, VEC>;
    GnChip<T, VEC> K(P, gn_smem, true);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32, threads = blockDim.x;
    float *part = K.red + 2 * K.nt * VEC;        // [threads] x 2
    float *csum = part + 2 * threads;            // [cb] x 2: channel sums of dz and dz xhat
    float *gsum = csum + 2 * K.cb;               // [gpc] x 2: their group sums times gamma
    float *k1 = gsum + 2 * P.gpc, *k2 = k1 + P.gpc;
    const int stride = K.nt * VEC;
    {
        const T *x = static_cast<const T *>(P.x.p) + K.n * P.x.sn + K.c + K.p0 * P.x.sp;
        const T *g = static_cast<const T *>(P.g.p) + K.n * P.g.sn + K.c + K.p0 * P.g.sp;
        const int64_t xstep = P.ty * P.x.sp, gstep = P.ty * P.g.sp;
        uint32_t xd = smem_u32(K.xs), gd = smem_u32(K.gs);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int end = K.quarter(k + 1);
            for (int i = K.quarter(k); i < end; ++i) {
                gn_copy_async<K.kBytes>(xd, x);
                gn_copy_async<K.kBytes>(gd, g);
                x += xstep;
                g += gstep;
                xd += stride * sizeof(T);
                gd += stride * sizeof(T);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }
    GnSlope<VEC> S;
    S.template load<UNI>(P, K.n, 0, K.c, K.c, K.on);
    float sa[VEC] = {}, sb[VEC] = {};
    T *xs = K.xs, *gs = K.gs;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (k == 0) gn_copy_wait<3>();
        if (k == 1) gn_copy_wait<2>();
        if (k == 2) gn_copy_wait<1>();
        if (k == 3) gn_copy_wait<0>();
        const int end = K.quarter(k + 1);
#pragma unroll 1
        for (int i = K.quarter(k); i < end; ++i, xs += stride, gs += stride) {
            float xv[VEC], gv[VEC];
            V::widen(V::load(xs), xv);
            V::widen(V::load(gs), gv);
            S.apply(P.act, xv, gv);
            add_to(sa, gv);
            fma_to(sb, gv, xv, sb);
            if constexpr (sizeof(T) == 4) {   // xhat and dz in the slots: not computed again
                V::store(xs, xv);
                V::store(gs, gv);
            }
        }
    }
    channel_sums<VEC>(P, K.red, part, csum, K.on, sa, sb);
    gamma_sums(P, csum, K.cb, K.chunk * K.cb, P.D, [&](int g, float s, float t) {
        gsum[g] = s;
        gsum[P.gpc + g] = t;
    });
    K.meet();
    const float total = static_cast<float>(P.HW) * P.D;
    for (int g = warp; g < 2 * P.gpc; g += warps) {
        float s = gsum[g];
        if (P.splits > 1) s = warp_sum_f(lane < P.splits ? gn_ld_rank(gsum + g, lane) : 0.f, 8);
        if (lane == 0) k1[g] = s / total;        // k2 follows k1
    }
    // the image's channel sums, for ggamma and gbeta: each CTA its share
    float *out = P.part + static_cast<int64_t>(K.n) * 2 * P.C + K.chunk * K.cb;
    for (int ch = threadIdx.x * P.splits + K.rank; ch < K.cb; ch += threads * P.splits) {
        float s = 0.f, t = 0.f;
        if (P.splits == 1) {
            s = csum[ch];
            t = csum[K.cb + ch];
        } else {
            for (int r = 0; r < P.splits; r += 2) {   // an even number of CTAs
                const float s0 = gn_ld_rank(csum + ch, r), s1 = gn_ld_rank(csum + ch, r + 1);
                const float t0 = gn_ld_rank(csum + K.cb + ch, r), t1 = gn_ld_rank(csum + K.cb + ch, r + 1);
                s += s0 + s1;
                t += t0 + t1;
            }
        }
        out[ch] = s;
        out[P.C + ch] = t;
    }
    if (P.splits > 1) gn_cluster_arrive();
    __syncthreads();
    // gx = rstd gamma dz - (rstd k1 + xhat rstd k2); sa, sb: the last two
    float scale[VEC];
    per_channel_group<VEC, UNI>(K.col * VEC, P.D, [&](int q, int g) {
        scale[q] = S.rstd[q] * S.gamma[q];
        sa[q] = -S.rstd[q] * k1[g];
        sb[q] = -S.rstd[q] * k2[g];
    });
    T *o = static_cast<T *>(P.out) + K.n * P.on + K.c + K.p0 * P.op;
    const int64_t step = P.ty * P.op;
    xs = K.xs;
    gs = K.gs;
#pragma unroll 1
    for (int i = 0; i < K.count; ++i, xs += stride, gs += stride, o += step) {
        float xv[VEC], gv[VEC];
        V::widen(V::load(xs), xv);
        V::widen(V::load(gs), gv);
        if constexpr (sizeof(T) != 4) S.apply(P.act, xv, gv);
        fma_to(xv, xv, sb, sa);
        fma_to(gv, gv, scale, xv);
        V::store(o, gv);
    }
    if (P.splits > 1) gn_cluster_wait();
}

}  // namespace mqc
