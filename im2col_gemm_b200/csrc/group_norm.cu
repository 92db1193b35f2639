// group_norm.cu -- entry points of the group norm (include/mqc.h): argument
// checks, the split of the work, and the launches of group_norm.cuh.
#include "group_norm.cuh"

#include <algorithm>
#include <atomic>
#include <cstring>

#include "host.h"

namespace mqc {
namespace {

mqc_status check_tensor(const char *name, const char *what, const void *p, const mqc_t4 *d, const mqc_t4 *like) {
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

// Elements of one access: the most, up to 16 bytes, that divides the channels
// and every stride.
int vector_of(int32_t dtype, const mqc_t4 *const *d, int count) {
    int64_t bits = d[0]->d1;
    for (int i = 0; i < count; ++i) {
        if (d[i]->d2 * int64_t(d[i]->d3) > 1) bits |= d[i]->d3 > 1 ? d[i]->s3 : d[i]->s2;
        if (d[i]->d0 > 1) bits |= d[i]->s0;
    }
    int v = 16 / dtype_bytes(dtype);
    while (bits % v != 0) v /= 2;
    return v;
}

// The split of a tensor into blocks: channel vectors along tx, pixels along
// ty, and pixel slabs so that there are about 16 blocks an SM (148 of them)
// while a thread still has at least four pixels.
void split(GnParams &P, int vec) {
    const int64_t cv = P.C / vec;
    P.tx = static_cast<int32_t>(std::min<int64_t>(cv, kGnThreads));
    P.ty = kGnThreads / P.tx;
    P.col_blocks = static_cast<int32_t>(ceil_div(cv, P.tx));
    const int64_t want = std::max<int64_t>(1, 148 * 16 / std::max<int64_t>(1, int64_t(P.N) * P.col_blocks));
    const int64_t most = ceil_div(P.HW, int64_t(P.ty) * 4);
    P.slab = static_cast<int32_t>(ceil_div(P.HW, std::min(want, most)));
    P.slabs = static_cast<int32_t>(ceil_div(P.HW, P.slab));
}

GnTensor tensor_of(const void *p, const mqc_t4 *d) {
    return GnTensor{p, d->d0 > 1 ? d->s0 : 0, d->d3 > 1 ? d->s3 : d->s2};
}

// Shared memory of the on-chip form besides the slots: row sums, 256 partial
// sums, two channel sums, four group sums, and the slots' alignment.
int64_t chip_extra(int tx, int ty, int vec, int gpc) {
    return 16 + 4 * (int64_t(tx) * ty * vec + kGnThreads + 2 * int64_t(tx) * vec + 4 * int64_t(gpc));
}
constexpr int64_t kChipSmem = 200 * 1024;

// The on-chip form of a tensor, if a cluster of at most eight CTAs holds one
// image's chunk of channels: the chunk (whole groups, whole vectors) and the
// number of CTAs with the least estimated time, in ns: the busiest SM's bytes
// at its share of the memory bandwidth (43 bytes/ns; rows below 32 bytes waste
// sectors), and for each round of resident CTAs the latency of loads and
// barriers, half hidden when several CTAs share an SM.
bool search_chip(GnParams &P, int vec, int32_t dtype, bool bwd, int64_t &smem) {
    const int size = dtype_bytes(dtype);
    if (vec * size < 4) return false;
    double best = 1e300;
    for (int gpc = 1; gpc <= P.G; ++gpc) {
        if (P.G % gpc != 0 || (int64_t(gpc) * P.D) % vec != 0) continue;
        const int64_t tx = int64_t(gpc) * P.D / vec;
        if (tx > kGnThreads) break;
        const int ty = static_cast<int>(kGnThreads / tx);
        const int64_t row = int64_t(gpc) * P.D * size;
        for (int splits = 1; splits <= 8; splits *= 2) {
            const int64_t slab = ceil_div(P.HW, splits), iters = ceil_div(slab, ty);
            const int64_t need = iters * tx * ty * vec * size * (bwd ? 2 : 1) +
                                 chip_extra(static_cast<int>(tx), ty, vec, gpc);
            if (need > kChipSmem || (splits > 1 && slab * (splits - 1) >= P.HW)) continue;
            const int64_t ctas = int64_t(P.N) * (P.G / gpc) * splits;
            const int64_t resident = std::min<int64_t>(4, (228 * 1024) / (need + 1024));
            const double waste = row < 32 ? 32.0 / row : (row < 64 ? 1.1 : 1.0);
            const double moved = double(slab) * row * (bwd ? 3 : 2) * waste;
            const double ns = ceil_div(ctas, 148) * moved / 43.0 +
                              ceil_div(ctas, 148 * resident) * (resident > 1 ? 1500.0 : 3000.0) + (splits > 1 ? 500.0 : 0.0);
            if (ns < best) {
                best = ns;
                P.gpc = gpc;
                P.chunks = P.G / gpc;
                P.tx = static_cast<int32_t>(tx);
                P.ty = ty;
                P.splits = splits;
                P.slab = static_cast<int32_t>(slab);
                P.iters = static_cast<int32_t>(iters);
                smem = need;
            }
        }
    }
    return best < 1e300;
}

// The same, remembered by sizes (the search takes some microseconds).
bool plan_chip(GnParams &P, int vec, int32_t dtype, bool bwd, int64_t &smem) {
    struct Entry {
        int32_t key[7], plan[7];
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
        const int32_t plan[7] = {P.gpc, P.chunks, P.tx, P.ty, P.splits, P.slab, P.iters};
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
    smem = e.smem;
    return e.found;
}

// Workspace of a call: per-channel partial sums of every slab (one for the
// gradients of the on-chip form), and the gradient's two coefficients a group.
size_t part_bytes(GnParams P, int vec, int32_t dtype, bool bwd, bool &chip) {
    int64_t smem;
    if ((chip = plan_chip(P, vec, dtype, bwd, smem))) {
        if (!bwd) return 0;
        P.slabs = 1;
    } else {
        split(P, vec);
    }
    return static_cast<size_t>(round_up(int64_t(P.N) * P.slabs * 2 * P.C * 4, 256));
}
size_t workspace_bytes(const GnParams &P, int vec, int32_t dtype, bool bwd) {
    bool chip;
    const size_t n = part_bytes(P, vec, dtype, bwd, chip);
    return n + (bwd && !chip ? static_cast<size_t>(round_up(int64_t(P.N) * P.G * 8, 256)) : 0);
}

template <typename T, int VEC>
mqc_status launch(GnParams &P, int32_t dtype, bool bwd, const DeviceLimits &d, cudaStream_t s) {
    const int64_t cb = P.ggamma || P.gbeta ? ceil_div(P.C, 32) : 0;
    int64_t smem = 0;
    if constexpr (VEC * sizeof(T) >= 4)
        if (plan_chip(P, VEC, dtype, bwd, smem)) {
            void (*kernel)(GnParams) = bwd ? gn_chip_bwd_kernel<T, VEC> : gn_chip_fwd_kernel<T, VEC>;
            static std::atomic<bool> allowed[2][64];
            if (!allowed[bwd][d.device].load(std::memory_order_acquire)) {
                cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize, kChipSmem);
                if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(group norm)");
                allowed[bwd][d.device].store(true, std::memory_order_release);
            }
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(static_cast<unsigned>(int64_t(P.N) * P.chunks * P.splits));
            cfg.blockDim = dim3(kGnThreads);
            cfg.dynamicSmemBytes = static_cast<size_t>(smem);
            cfg.stream = s;
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = P.splits;
            at[0].val.clusterDim.y = 1;
            at[0].val.clusterDim.z = 1;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P);
            if (e != cudaSuccess) return cuda_fail(e, "group norm launch");
            if (bwd && cb > 0) {
                P.slabs = 1;
                gn_bwd_finish_kernel<<<static_cast<unsigned>(cb), 128, 0, s>>>(P, 0);
                e = cudaGetLastError();
                if (e != cudaSuccess) return cuda_fail(e, "group norm launch");
            }
            return MQC_OK;
        }
    split(P, VEC);
    const unsigned grid = static_cast<unsigned>(int64_t(P.N) * P.slabs * P.col_blocks);
    const unsigned gb = static_cast<unsigned>(ceil_div(int64_t(P.N) * P.G, 4));
    if (bwd) {
        gn_bwd_sums_kernel<T, VEC><<<grid, kGnThreads, 0, s>>>(P);
        gn_bwd_finish_kernel<<<gb + static_cast<unsigned>(cb), 128, 0, s>>>(P, static_cast<int32_t>(gb));
        gn_bwd_apply_kernel<T, VEC><<<grid, kGnThreads, 0, s>>>(P);
    } else {
        gn_stats_kernel<T, VEC><<<grid, kGnThreads, 0, s>>>(P);
        gn_finish_kernel<<<gb, 128, 0, s>>>(P);
        gn_apply_kernel<T, VEC><<<grid, kGnThreads, 0, s>>>(P);
    }
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MQC_OK : cuda_fail(e, "group norm launch");
}

template <typename T>
mqc_status launch_vec(GnParams &P, int vec, int32_t dtype, bool bwd, const DeviceLimits &d, cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (vec == 8) return launch<T, 8>(P, dtype, bwd, d, s);
    if (vec == 4) return launch<T, 4>(P, dtype, bwd, d, s);
    if (vec == 2) return launch<T, 2>(P, dtype, bwd, d, s);
    return launch<T, 1>(P, dtype, bwd, d, s);
}

mqc_status check_workspace(const char *name, const void *ws, size_t bytes, size_t need) {
    if (need == 0) return MQC_OK;
    if (ws == nullptr || bytes < need)
        return fail(MQC_ERR_WORKSPACE, "%s: needs %zu workspace bytes, got %zu", name, need, ws ? bytes : size_t(0));
    if (!aligned16(ws)) return fail(MQC_ERR_ALIGNMENT, "%s: workspace not 16-byte aligned", name);
    return MQC_OK;
}

mqc_status run(const char *name, GnParams &P, int vec, int32_t dtype, bool bwd, cudaStream_t s) {
    // every grid below has at most this many blocks
    if (int64_t(P.N) * P.G * 8 > (int64_t(1) << 31) - 1 || int64_t(P.N) * P.C > (int64_t(1) << 31) - 1)
        return fail(MQC_ERR_INVALID, "%s: tensor too large", name);
    DeviceLimits d;
    mqc_status st = device_limits(&d);
    if (st != MQC_OK) return st;
    if (dtype == MQC_F32) return launch_vec<float>(P, vec, dtype, bwd, d, s);
    if (dtype == MQC_BF16) return launch_vec<__nv_bfloat16>(P, vec, dtype, bwd, d, s);
    return launch_vec<__half>(P, vec, dtype, bwd, d, s);
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
    return workspace_bytes(P, vector_of(dtype, all, 2), dtype, false);
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
    return workspace_bytes(P, vector_of(dtype, all, 3), dtype, true);
}

mqc_status mqc_group_norm_fwd(const void *x, const mqc_t4 *xd, int32_t dtype, const float *gamma, const float *beta,
                              int32_t groups, float eps, int32_t act, void *y, const mqc_t4 *yd, float *mean,
                              float *rstd, void *workspace, size_t workspace_bytes, void *stream) {
    const char *name = "group_norm_fwd";
    mqc_status st = check_extents(name, xd, dtype, groups, act);
    if (st != MQC_OK) return st;
    if (!(eps >= 0.f)) return fail(MQC_ERR_INVALID, "%s: eps must not be negative", name);
    if (xd->d0 == 0) return MQC_OK;
    if ((st = check_tensor(name, "x", x, xd, xd)) != MQC_OK) return st;
    if ((st = check_tensor(name, "y", y, yd, xd)) != MQC_OK) return st;
    if (mean == nullptr || rstd == nullptr) return fail(MQC_ERR_INVALID, "%s: null statistics", name);
    GnParams P{};
    fill(P, xd, groups);
    const mqc_t4 *all[2] = {xd, yd};
    const int vec = vector_of(dtype, all, 2);
    const size_t need = mqc::workspace_bytes(P, vec, dtype, false);
    if ((st = check_workspace(name, workspace, workspace_bytes, need)) != MQC_OK) return st;
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
    P.part = static_cast<float *>(workspace);
    return run(name, P, vec, dtype, false, static_cast<cudaStream_t>(stream));
}

mqc_status mqc_group_norm_bwd(const void *g, const mqc_t4 *gd, const void *x, const mqc_t4 *xd, int32_t dtype,
                              const float *gamma, const float *beta, const float *mean, const float *rstd,
                              int32_t groups, int32_t act, void *gx, const mqc_t4 *gxd, float *ggamma, float *gbeta,
                              void *workspace, size_t workspace_bytes, void *stream) {
    const char *name = "group_norm_bwd";
    mqc_status st = check_extents(name, xd, dtype, groups, act);
    if (st != MQC_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (xd->d0 == 0) {
        cudaError_t e = cudaSuccess;
        if (ggamma) e = cudaMemsetAsync(ggamma, 0, size_t(xd->d1) * 4, s);
        if (e == cudaSuccess && gbeta) e = cudaMemsetAsync(gbeta, 0, size_t(xd->d1) * 4, s);
        return e == cudaSuccess ? MQC_OK : cuda_fail(e, "group_norm_bwd memset");
    }
    if ((st = check_tensor(name, "x", x, xd, xd)) != MQC_OK) return st;
    if ((st = check_tensor(name, "g", g, gd, xd)) != MQC_OK) return st;
    if ((st = check_tensor(name, "gx", gx, gxd, xd)) != MQC_OK) return st;
    if (mean == nullptr || rstd == nullptr) return fail(MQC_ERR_INVALID, "%s: null statistics", name);
    GnParams P{};
    fill(P, xd, groups);
    const mqc_t4 *all[3] = {xd, gd, gxd};
    const int vec = vector_of(dtype, all, 3);
    const size_t need = mqc::workspace_bytes(P, vec, dtype, true);
    if ((st = check_workspace(name, workspace, workspace_bytes, need)) != MQC_OK) return st;
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
    bool chip;
    P.coef = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + part_bytes(P, vec, dtype, true, chip));
    return run(name, P, vec, dtype, true, s);
}

}  // extern "C"
