// group_norm.cu -- entry points of the group norm (include/mqc.h): argument
// checks, the split of the work, and the launches of group_norm.cuh.
#include "group_norm.cuh"

#include <algorithm>
#include <atomic>
#include <cstring>

#include "host.h"

namespace mqc {
namespace {

mqc_status check_tensor(const char *name, const char *what, const void *p, const mqc_t4 *d, const mqc_t4 *like,
                        bool written) {
    if (p == nullptr || d == nullptr) return fail(MQC_ERR_INVALID, "%s: %s or its descriptor is null", name, what);
    if (d->d0 != like->d0 || d->d1 != like->d1 || d->d2 != like->d2 || d->d3 != like->d3)
        return fail(MQC_ERR_INVALID, "%s: the extents of %s differ", name, what);
    if (!aligned16(p)) return fail(MQC_ERR_ALIGNMENT, "%s: %s not 16-byte aligned", name, what);
    const bool many_c = d->d1 > 1, many_w = d->d3 > 1, many_h = d->d2 > 1;
    const int64_t sp = many_w ? d->s3 : d->s2;   // pixel stride
    if ((many_c && d->s1 != 1) || (many_w && many_h && d->s2 != d->s3 * d->d3))
        return fail(MQC_ERR_UNSUPPORTED, "%s: %s must be channels last (channel stride 1, rows of pixels in sequence)",
                    name, what);
    if (((many_w || many_h) && sp < d->d1) || sp > (int64_t(1) << 38) || d->s0 < 0 || d->s0 > (int64_t(1) << 44))
        return fail(MQC_ERR_UNSUPPORTED, "%s: strides of %s out of range", name, what);
    // images one after another, or interleaved pixel by pixel
    const int64_t pixels = (int64_t(d->d2) * d->d3 - 1) * sp + d->d1, images = int64_t(d->d0 - 1) * d->s0 + d->d1;
    if (written && d->d0 > 1 && d->s0 < pixels && !(d->s0 >= d->d1 && sp >= images))
        return fail(MQC_ERR_UNSUPPORTED, "%s: the images of %s overlap", name, what);
    return MQC_OK;
}

// fp32 parameters and statistics, NULL allowed.
mqc_status check_params(const char *name, const float *const *p, int count) {
    for (int i = 0; i < count; ++i)
        if ((reinterpret_cast<uintptr_t>(p[i]) & 3u) != 0)
            return fail(MQC_ERR_ALIGNMENT, "%s: parameters and statistics must be 4-byte aligned", name);
    return MQC_OK;
}

mqc_status check_extents(const char *name, const mqc_t4 *d, int32_t dtype, int32_t groups, int32_t act) {
    if (d == nullptr) return fail(MQC_ERR_INVALID, "%s: null descriptor", name);
    if (dtype != MQC_F32 && dtype != MQC_BF16 && dtype != MQC_F16) return fail(MQC_ERR_INVALID, "%s: bad dtype", name);
    if (d->d0 < 0 || d->d1 <= 0 || d->d2 <= 0 || d->d3 <= 0) return fail(MQC_ERR_INVALID, "%s: bad extents", name);
    if (groups <= 0 || d->d1 % groups != 0)
        return fail(MQC_ERR_INVALID, "%s: %d groups do not divide %d channels", name, groups, d->d1);
    if (!act_ok(act)) return fail(MQC_ERR_INVALID, "%s: bad activation", name);
    if (int64_t(d->d2) * d->d3 > (int64_t(1) << 30)) return fail(MQC_ERR_INVALID, "%s: too many pixels", name);
    return MQC_OK;
}

// Elements of one access: the most, up to `most` and 16 bytes, that divides the
// channels and every stride.  (Backward four: eight channels' constants and
// sums take 128 registers, and the fewer warps cost more than the wider loads
// gain.)
int vector_of(int32_t dtype, const mqc_t4 *const *d, int count, int most) {
    int64_t bits = d[0]->d1;
    for (int i = 0; i < count; ++i) {
        if (d[i]->d2 * int64_t(d[i]->d3) > 1) bits |= d[i]->d3 > 1 ? d[i]->s3 : d[i]->s2;
        if (d[i]->d0 > 1) bits |= d[i]->s0;
    }
    int v = std::min(most, 16 / dtype_bytes(dtype));
    while (bits % v != 0) v /= 2;
    return v;
}

GnTensor tensor_of(const void *p, const mqc_t4 *d) {
    return GnTensor{p, d->d0 > 1 ? d->s0 : 0, d->d3 > 1 ? d->s3 : d->s2};
}

// Sums that a thread leaves for the groups of its vector: one when the vector
// lies in one group, one a group when groups tile the vector, else one a
// channel.
int sums_left(int D, int vec) { return D % vec == 0 ? 1 : (vec % D == 0 ? vec / D : vec); }

// Shared memory of the on-chip form besides the slots (and their alignment):
// row sums, group sums; backward also a partial and a channel sum, all twice.
int64_t chip_extra(int64_t tx, int64_t ty, int vec, int D, int64_t gpc, int threads, bool bwd) {
    return 16 + 4 * (bwd ? 2 * tx * ty * vec + 2 * threads + 2 * tx * vec + 4 * gpc
                         : tx * ty * sums_left(D, vec) + 4 * gpc);
}
constexpr int kChipSmem = 200 * 1024;

// The on-chip form of a tensor, if a cluster of at most 16 CTAs holds one
// image's chunk of channels: the chunk (whole groups, whole vectors), threads
// and CTAs of the least estimated time.  In ns, for one round of the CTAs that
// an SM holds at once: their loads at the SM's share of the memory bandwidth
// (43 bytes/ns; rows below 64 bytes waste half of it), then the larger of
// their stores and their arithmetic (about 14 warp instructions an element
// forward, 26 backward, and 300 a thread for constants and sums, at 0.16 a
// cycle for each warp of a scheduler, up to 0.75), and the latency of loads
// and barriers.
bool search_chip(GnParams &P, int vec, int32_t dtype, bool bwd, int64_t &smem) {
    const int size = dtype_bytes(dtype);
    if (vec * size < 4) return false;
    double best = 1e300;
    for (int gpc = 1; gpc <= P.G; ++gpc) {
        if (P.G % gpc != 0 || (int64_t(gpc) * P.D) % vec != 0) continue;
        const int64_t tx = int64_t(gpc) * P.D / vec;
        if (tx > kGnThreads) break;
        const int64_t row = int64_t(gpc) * P.D * size;
        const double waste = row < 64 ? std::min(4.0, 96.0 / row) / 1.5 : 1.0;
        for (int threads = kGnThreads; threads >= 128 && threads >= tx; threads /= 2) {
            const int ty = static_cast<int>(threads / tx);
            for (int splits = 1; splits <= 16; splits *= 2) {
                const int64_t slab = ceil_div(P.HW, splits), iters = ceil_div(slab, ty);
                const int64_t need = iters * tx * ty * vec * size * (bwd ? 2 : 1) +
                                     chip_extra(tx, ty, vec, P.D, gpc, threads, bwd);
                if (need > kChipSmem || slab * (splits - 1) >= P.HW) continue;
                const int64_t ctas = int64_t(P.N) * (P.G / gpc) * splits;
                const int64_t resident = std::max<int64_t>(
                    1, std::min({ceil_div(ctas, 148), int64_t(1024 / threads), (228 * 1024) / (need + 1024)}));
                const double bytes = resident * double(slab) * row * waste / 43.0;
                const double warps = resident * threads / 128.0;
                const double issued = warps * (300.0 + iters * vec * (bwd ? 26.0 : 14.0)) /
                                      (1.9 * std::min(0.75, 0.16 * warps));
                const double round = bytes * (bwd ? 2 : 1) + std::max(bytes, issued) + (splits > 1 ? 3000.0 : 1800.0);
                const double ns = std::max(1.0, double(ctas) / (148 * resident)) * round;
                if (ns < best) {
                    best = ns;
                    P.gpc = gpc;
                    P.chunks = P.G / gpc;
                    P.tx = static_cast<int32_t>(tx);
                    P.ty = ty;
                    P.threads = threads;
                    P.splits = splits;
                    P.slab = static_cast<int32_t>(slab);
                    P.iters = static_cast<int32_t>(iters);
                    smem = need;
                }
            }
        }
    }
    return best < 1e300;
}

// The same, remembered by sizes (the search takes some microseconds).
bool plan_chip(GnParams &P, int vec, int32_t dtype, bool bwd, int64_t &smem) {
    struct Entry {
        int32_t key[7], plan[8];
        int64_t smem;
        bool used, found;
    };
    static thread_local Entry cache[16];
    const int32_t key[7] = {P.N, P.C, P.G, P.HW, vec, dtype, bwd ? 1 : 0};
    uint32_t h = 2166136261u;
    for (int32_t k : key) h = (h ^ static_cast<uint32_t>(k)) * 16777619u;
    Entry &e = cache[(h >> 16) % 16];
    if (!e.used || memcmp(e.key, key, sizeof key) != 0) {
        e.found = search_chip(P, vec, dtype, bwd, smem);
        memcpy(e.key, key, sizeof key);
        const int32_t plan[8] = {P.gpc, P.chunks, P.tx, P.ty, P.splits, P.slab, P.iters, P.threads};
        memcpy(e.plan, plan, sizeof plan);
        e.smem = smem;
        e.used = true;
        return e.found;
    }
    P.gpc = e.plan[0];
    P.chunks = e.plan[1];
    P.tx = e.plan[2];
    P.ty = e.plan[3];
    P.splits = e.plan[4];
    P.slab = e.plan[5];
    P.iters = e.plan[6];
    P.threads = e.plan[7];
    smem = e.smem;
    return e.found;
}

// The two-pass form: chunks of whole groups and whole vectors, about 512 bytes
// wide, or pieces of a group wider than a block; slabs of pixels so that all
// blocks (three on each of 148 SMs) run at once, while a thread still has
// eight pixels: a warp spends some 850 instructions on its place and its sums,
// 24 on a vector.  Returns the elements of a vector.
int plan_passes(GnParams &P, int vec, int32_t dtype) {
    int unit;   // groups that are whole vectors
    for (;; vec /= 2) {
        unit = 1;
        while ((int64_t(unit) * P.D) % vec != 0) ++unit;
        if (int64_t(unit) * P.D / vec <= kPassThreads || P.D % vec == 0) break;
    }
    P.splits = 0;
    if (int64_t(unit) * P.D / vec > kPassThreads) {   // unit = 1
        P.gpc = 1;
        P.width = kPassThreads * vec;
        P.pieces = static_cast<int32_t>(ceil_div(P.D, P.width));
        P.chunks = P.G * P.pieces;
    } else {
        P.gpc = unit;
        for (int g = unit; g <= P.G && int64_t(g) * P.D * dtype_bytes(dtype) <= 512; g += unit)
            if (P.G % g == 0) P.gpc = g;
        P.pieces = 1;
        P.width = P.gpc * P.D;
        P.chunks = P.G / P.gpc;
    }
    P.tx = P.width / vec;
    P.threads = kPassThreads;
    P.ty = P.threads / P.tx;
    const int64_t want = std::max<int64_t>(1, 148 * 3 / std::max<int64_t>(1, int64_t(P.N) * P.chunks));
    const int64_t most = ceil_div(P.HW, int64_t(P.ty) * 8);
    P.slab = static_cast<int32_t>(ceil_div(P.HW, std::min(want, most)));
    P.slabs = static_cast<int32_t>(ceil_div(P.HW, P.slab));
    return vec;
}

// The plan of a call and its workspace: backward, the channels' partial sums of
// every slab (one an image on chip); in two passes, the groups' too.
struct GnPlan {
    int vec;
    bool chip;
    int64_t smem, part, gpart;
    int64_t bytes() const { return part + gpart; }
};
GnPlan make_plan(GnParams &P, int vec, int32_t dtype, bool bwd) {
    GnPlan p{vec, false, 0, 0, 0};
    p.chip = plan_chip(P, vec, dtype, bwd, p.smem);
    // On chip a tensor is read once, but a CTA's phases overlap with nobody's
    // when it takes most of an SM, and clusters of many CTAs fill the chip in
    // fewer, longer rounds; two passes of small blocks overlap better, and the
    // second one finds what the first read last in L2.  From 118 shapes of 4 to
    // 380 MB, the slower form within 16% wherever this rule picks it; e.g. bf16
    // forward, on chip against two passes: 24x512x20x20 (one CTA) 8.3, 12.0 us;
    // 8x128x80x80 (four) 11.3, 16.3; 24x128x80x80 27.9, 27.2; 8x64x160x160
    // (16) 27.8, 19.7; backward 24x512x20x20 15.1, 17.7; 24x256x40x40 (two)
    // 35.5, 24.5; 8x128x80x80 (16) 28.0, 20.1.
    const int64_t bytes = int64_t(P.N) * P.C * P.HW * dtype_bytes(dtype) * (bwd ? 3 : 2);
    if (bwd ? P.splits > 4 || bytes > (int64_t(32) << 20) : P.splits > 2 && bytes * P.splits > 200000000)
        p.chip = false;
    if (p.chip) {
        P.slabs = 1;
        P.pieces = 1;
        P.width = P.tx * vec;
    } else {
        p.vec = plan_passes(P, vec, dtype);
        p.gpart = round_up(int64_t(P.N) * P.slabs * P.chunks * P.gpc * 8, 256);
    }
    if (bwd) p.part = round_up(int64_t(P.N) * P.slabs * 2 * P.C * 4, 256);
    const int cb = P.tx * p.vec;
    const bool uni = P.D % p.vec == 0;
    P.seg = bwd ? std::max(1, P.threads / cb) : sums_left(P.D, p.vec);
    P.fd_tx = make_fastdiv(P.tx);
    P.fd_ty = make_fastdiv(P.ty);
    P.fd_chunks = make_fastdiv(P.chunks);
    P.fd_slabs = make_fastdiv(P.slabs);
    P.fd_cb = make_fastdiv(cb);
    P.fd_entries = make_fastdiv(uni ? (P.pieces > 1 ? P.tx : P.D / p.vec) : (P.seg == p.vec ? P.D : 1));
    return p;
}

template <typename T, int VEC, bool UNI, bool BWD>
mqc_status launch(GnParams &P, const GnPlan &plan, const DeviceLimits &d, cudaStream_t s) {
    const int channel_blocks = BWD && (P.ggamma || P.gbeta) ? static_cast<int>(ceil_div(P.C, 32)) : 0;
    if constexpr (VEC * sizeof(T) >= 4)
        if (plan.chip) {
            void (*kernel)(GnParams);
            if constexpr (BWD) kernel = gn_chip_bwd_kernel<T, VEC, UNI>;
            else kernel = gn_chip_fwd_kernel<T, VEC, UNI>;
            static std::atomic<bool> allowed[64];
            if (!allowed[d.device].load(std::memory_order_acquire)) {
                cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize, kChipSmem);
                if (e == cudaSuccess)
                    e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
                if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(group norm)");
                allowed[d.device].store(true, std::memory_order_release);
            }
            const Launch chip(int64_t(P.N) * P.chunks * P.splits, P.threads, P.splits, plan.smem, false, s);
            cudaError_t e = cudaLaunchKernelEx(&chip.cfg, kernel, P);
            if (e != cudaSuccess) return cuda_fail(e, "group norm launch");
            if (channel_blocks > 0) {
                const Launch channels(channel_blocks, kGnThreads, 0, 0, true, s);
                e = cudaLaunchKernelEx(&channels.cfg, gn_channels_kernel, P, int64_t(P.N));
                if (e != cudaSuccess) return cuda_fail(e, "group norm launch");
            }
            return MQC_OK;
        }
    const unsigned grid = static_cast<unsigned>(int64_t(P.N) * P.slabs * P.chunks);
    const size_t nt = size_t(P.tx) * P.ty, groups = 2 * size_t(P.gpc) * 4;
    cudaError_t e;
    if constexpr (BWD) {
        P.channel_blocks = channel_blocks;
        const size_t ring = GnRing<T, VEC, 2>::kSlotBytes;
        const size_t sums = 4 * (2 * nt * VEC + 2 * P.threads + 2 * size_t(P.tx) * VEC);
        const size_t join = P.threads / 32 * 2 * 32 * 8;
        gn_bwd_sums_kernel<T, VEC, UNI><<<grid, P.threads, std::max(ring, sums), s>>>(P);
        const Launch apply(int64_t(grid) + channel_blocks, P.threads, 0, std::max(ring + kJoinBytes + groups, join), true, s);
        e = cudaGetLastError();
        if (e == cudaSuccess) e = cudaLaunchKernelEx(&apply.cfg, gn_bwd_apply_kernel<T, VEC, UNI>, P);
    } else {
        const size_t ring = GnRing<T, VEC, 1>::kSlotBytes;
        const size_t sums = 4 * nt * (UNI ? 1 : P.seg) + groups;
        gn_stats_kernel<T, VEC, UNI><<<grid, P.threads, std::max(ring, sums), s>>>(P);
        const Launch apply(grid, P.threads, 0, ring + kJoinBytes + groups, true, s);
        e = cudaGetLastError();
        if (e == cudaSuccess) e = cudaLaunchKernelEx(&apply.cfg, gn_apply_kernel<T, VEC, UNI>, P);
    }
    return e == cudaSuccess ? MQC_OK : cuda_fail(e, "group norm launch");
}

template <typename T, bool BWD>
mqc_status launch_vec(GnParams &P, const GnPlan &plan, const DeviceLimits &d, cudaStream_t s) {
    const bool uni = P.D % plan.vec == 0;   // always, with one channel a vector
    if constexpr (sizeof(T) == 2 && !BWD)
        if (plan.vec == 8) return uni ? launch<T, 8, true, BWD>(P, plan, d, s) : launch<T, 8, false, BWD>(P, plan, d, s);
    if (plan.vec == 4) return uni ? launch<T, 4, true, BWD>(P, plan, d, s) : launch<T, 4, false, BWD>(P, plan, d, s);
    if (plan.vec == 2) return uni ? launch<T, 2, true, BWD>(P, plan, d, s) : launch<T, 2, false, BWD>(P, plan, d, s);
    return launch<T, 1, true, BWD>(P, plan, d, s);
}
template <typename T>
mqc_status launch_dir(GnParams &P, const GnPlan &plan, bool bwd, const DeviceLimits &d, cudaStream_t s) {
    return bwd ? launch_vec<T, true>(P, plan, d, s) : launch_vec<T, false>(P, plan, d, s);
}

mqc_status check_workspace(const char *name, const void *ws, size_t bytes, size_t need) {
    if (need == 0) return MQC_OK;
    if (ws == nullptr || bytes < need)
        return fail(MQC_ERR_WORKSPACE, "%s: needs %zu workspace bytes, got %zu", name, need, ws ? bytes : size_t(0));
    if (!aligned16(ws)) return fail(MQC_ERR_ALIGNMENT, "%s: workspace not 16-byte aligned", name);
    return MQC_OK;
}

mqc_status run(const char *name, GnParams &P, const GnPlan &plan, int32_t dtype, bool bwd, cudaStream_t s) {
    // every grid above has at most this many blocks
    if (int64_t(P.N) * P.G * 16 > (int64_t(1) << 31) - 1 || int64_t(P.N) * P.slabs * P.chunks > (int64_t(1) << 30))
        return fail(MQC_ERR_INVALID, "%s: tensor too large", name);
    DeviceLimits d;
    mqc_status st = device_limits(&d);
    if (st != MQC_OK) return st;
    if (dtype == MQC_F32) return launch_dir<float>(P, plan, bwd, d, s);
    if (dtype == MQC_BF16) return launch_dir<__nv_bfloat16>(P, plan, bwd, d, s);
    return launch_dir<__half>(P, plan, bwd, d, s);
}

void fill(GnParams &P, const mqc_t4 *d, int32_t groups) {
    P.N = d->d0;
    P.C = d->d1;
    P.G = groups;
    P.D = d->d1 / groups;
    P.HW = d->d2 * d->d3;
}

}  // namespace
}  // namespace mqc

using namespace mqc;

extern "C" {

size_t mqc_group_norm_fwd_workspace_bytes(const mqc_t4 *xd, const mqc_t4 *yd, int32_t dtype, int32_t groups) {
    const char *name = "group_norm_fwd_workspace_bytes";
    if (check_extents(name, xd, dtype, groups, MQC_ACT_NONE) != MQC_OK || yd == nullptr || xd->d0 == 0) return 0;
    GnParams P{};
    fill(P, xd, groups);
    const mqc_t4 *all[2] = {xd, yd};
    return static_cast<size_t>(make_plan(P, vector_of(dtype, all, 2, 8), dtype, false).bytes());
}

size_t mqc_group_norm_bwd_workspace_bytes(const mqc_t4 *gd, const mqc_t4 *xd, const mqc_t4 *gxd, int32_t dtype,
                                          int32_t groups) {
    const char *name = "group_norm_bwd_workspace_bytes";
    if (check_extents(name, xd, dtype, groups, MQC_ACT_NONE) != MQC_OK || gd == nullptr || gxd == nullptr ||
        xd->d0 == 0)
        return 0;
    GnParams P{};
    fill(P, xd, groups);
    const mqc_t4 *all[3] = {xd, gd, gxd};
    return static_cast<size_t>(make_plan(P, vector_of(dtype, all, 3, 4), dtype, true).bytes());
}

mqc_status mqc_group_norm_fwd(const void *x, const mqc_t4 *xd, int32_t dtype, const float *gamma, const float *beta,
                              int32_t groups, float eps, int32_t act, void *y, const mqc_t4 *yd, float *mean,
                              float *rstd, void *workspace, size_t workspace_bytes, void *stream) {
    const char *name = "group_norm_fwd";
    mqc_status st = check_extents(name, xd, dtype, groups, act);
    if (st != MQC_OK) return st;
    if (!(eps >= 0.f)) return fail(MQC_ERR_INVALID, "%s: eps must not be negative", name);
    if (xd->d0 == 0) return MQC_OK;
    if ((st = check_tensor(name, "x", x, xd, xd, false)) != MQC_OK) return st;
    if ((st = check_tensor(name, "y", y, yd, xd, true)) != MQC_OK) return st;
    if (mean == nullptr || rstd == nullptr) return fail(MQC_ERR_INVALID, "%s: null statistics", name);
    const float *params[4] = {gamma, beta, mean, rstd};
    if ((st = check_params(name, params, 4)) != MQC_OK) return st;
    GnParams P{};
    fill(P, xd, groups);
    const mqc_t4 *all[2] = {xd, yd};
    const GnPlan plan = make_plan(P, vector_of(dtype, all, 2, 8), dtype, false);
    if ((st = check_workspace(name, workspace, workspace_bytes, plan.bytes())) != MQC_OK) return st;
    P.x = tensor_of(x, xd);
    const GnTensor o = tensor_of(y, yd);
    P.out = y;
    P.on = o.sn;
    P.op = o.sp;
    P.gamma = gamma;
    P.beta = beta;
    P.mean = mean;
    P.rstd = rstd;
    P.eps = eps;
    P.act = act;
    P.gpart = static_cast<float *>(workspace);
    return run(name, P, plan, dtype, false, static_cast<cudaStream_t>(stream));
}

mqc_status mqc_group_norm_bwd(const void *g, const mqc_t4 *gd, const void *x, const mqc_t4 *xd, int32_t dtype,
                              const float *gamma, const float *beta, const float *mean, const float *rstd,
                              int32_t groups, int32_t act, void *gx, const mqc_t4 *gxd, float *ggamma, float *gbeta,
                              void *workspace, size_t workspace_bytes, void *stream) {
    const char *name = "group_norm_bwd";
    mqc_status st = check_extents(name, xd, dtype, groups, act);
    if (st != MQC_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const float *params[6] = {gamma, beta, mean, rstd, ggamma, gbeta};
    if ((st = check_params(name, params, 6)) != MQC_OK) return st;
    if (xd->d0 == 0) {
        cudaError_t e = cudaSuccess;
        if (ggamma) e = cudaMemsetAsync(ggamma, 0, size_t(xd->d1) * 4, s);
        if (e == cudaSuccess && gbeta) e = cudaMemsetAsync(gbeta, 0, size_t(xd->d1) * 4, s);
        return e == cudaSuccess ? MQC_OK : cuda_fail(e, "group_norm_bwd memset");
    }
    if ((st = check_tensor(name, "x", x, xd, xd, false)) != MQC_OK) return st;
    if ((st = check_tensor(name, "g", g, gd, xd, false)) != MQC_OK) return st;
    if ((st = check_tensor(name, "gx", gx, gxd, xd, true)) != MQC_OK) return st;
    if (mean == nullptr || rstd == nullptr) return fail(MQC_ERR_INVALID, "%s: null statistics", name);
    GnParams P{};
    fill(P, xd, groups);
    const mqc_t4 *all[3] = {xd, gd, gxd};
    const GnPlan plan = make_plan(P, vector_of(dtype, all, 3, 4), dtype, true);
    if ((st = check_workspace(name, workspace, workspace_bytes, plan.bytes())) != MQC_OK) return st;
    P.x = tensor_of(x, xd);
    P.g = tensor_of(g, gd);
    const GnTensor o = tensor_of(gx, gxd);
    P.out = gx;
    P.on = o.sn;
    P.op = o.sp;
    P.gamma = gamma;
    P.beta = beta;
    P.mean = const_cast<float *>(mean);
    P.rstd = const_cast<float *>(rstd);
    P.ggamma = ggamma;
    P.gbeta = gbeta;
    P.act = act;
    P.part = static_cast<float *>(workspace);
    P.gpart = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + plan.part);
    return run(name, P, plan, dtype, true, s);
}

}  // extern "C"
