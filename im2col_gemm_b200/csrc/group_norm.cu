// group_norm.cu -- entry points of the group norm (include/mqc.h): argument
// checks, the split of the work, and the launches of group_norm.cuh.
#include "group_norm.cuh"

#include <algorithm>

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

// Upper bound over the vector sizes.
int64_t most_slabs(const mqc_t4 *d, int32_t dtype) {
    int64_t most = 1;
    for (int vec = 16 / dtype_bytes(dtype); vec >= 1; vec /= 2) {
        if (d->d1 % vec != 0) continue;
        GnParams P{};
        P.N = d->d0;
        P.C = d->d1;
        P.HW = d->d2 * d->d3;
        split(P, vec);
        most = std::max<int64_t>(most, P.slabs);
    }
    return most;
}

GnTensor tensor_of(const void *p, const mqc_t4 *d) {
    return GnTensor{p, d->d0 > 1 ? d->s0 : 0, d->d3 > 1 ? d->s3 : d->s2};
}

template <typename T, int VEC>
void launch_fwd(const GnParams &P, unsigned grid, cudaStream_t s) {
    gn_stats_kernel<T, VEC><<<grid, kGnThreads, 0, s>>>(P);
    gn_finish_kernel<<<static_cast<unsigned>(ceil_div(int64_t(P.N) * P.G, 4)), 128, 0, s>>>(P);
    gn_apply_kernel<T, VEC><<<grid, kGnThreads, 0, s>>>(P);
}

template <typename T, int VEC>
void launch_bwd(const GnParams &P, unsigned grid, cudaStream_t s) {
    gn_bwd_sums_kernel<T, VEC><<<grid, kGnThreads, 0, s>>>(P);
    const int64_t gb = ceil_div(int64_t(P.N) * P.G, 4);
    const int64_t cb = P.ggamma || P.gbeta ? ceil_div(P.C, 32) : 0;
    gn_bwd_finish_kernel<<<static_cast<unsigned>(gb + cb), 128, 0, s>>>(P, static_cast<int32_t>(gb));
    gn_bwd_apply_kernel<T, VEC><<<grid, kGnThreads, 0, s>>>(P);
}

template <typename T>
void launch(const GnParams &P, int vec, bool bwd, unsigned grid, cudaStream_t s) {
    constexpr int most = 16 / sizeof(T);
    if constexpr (most == 8)
        if (vec == 8) return bwd ? launch_bwd<T, 8>(P, grid, s) : launch_fwd<T, 8>(P, grid, s);
    if (vec == 4) return bwd ? launch_bwd<T, 4>(P, grid, s) : launch_fwd<T, 4>(P, grid, s);
    if (vec == 2) return bwd ? launch_bwd<T, 2>(P, grid, s) : launch_fwd<T, 2>(P, grid, s);
    return bwd ? launch_bwd<T, 1>(P, grid, s) : launch_fwd<T, 1>(P, grid, s);
}

mqc_status check_workspace(const char *name, const void *ws, size_t bytes, size_t need) {
    if (ws == nullptr || bytes < need)
        return fail(MQC_ERR_WORKSPACE, "%s: needs %zu workspace bytes, got %zu", name, need, ws ? bytes : size_t(0));
    if (!aligned16(ws)) return fail(MQC_ERR_ALIGNMENT, "%s: workspace not 16-byte aligned", name);
    return MQC_OK;
}

mqc_status run(const char *name, GnParams &P, int vec, int32_t dtype, bool bwd, cudaStream_t s) {
    split(P, vec);
    const int64_t grid = int64_t(P.N) * P.slabs * P.col_blocks;
    if (grid > (int64_t(1) << 31) - 1 || int64_t(P.N) * P.G > (int64_t(1) << 31))
        return fail(MQC_ERR_INVALID, "%s: tensor too large", name);
    DeviceLimits d;
    mqc_status st = device_limits(&d);
    if (st != MQC_OK) return st;
    if (dtype == MQC_F32) launch<float>(P, vec, bwd, static_cast<unsigned>(grid), s);
    else if (dtype == MQC_BF16) launch<__nv_bfloat16>(P, vec, bwd, static_cast<unsigned>(grid), s);
    else launch<__half>(P, vec, bwd, static_cast<unsigned>(grid), s);
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MQC_OK : cuda_fail(e, "group norm launch");
}

size_t part_bytes(const mqc_t4 *d, int32_t dtype) {
    return static_cast<size_t>(round_up(int64_t(d->d0) * most_slabs(d, dtype) * 2 * d->d1 * 4, 256));
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

size_t mqc_group_norm_workspace_bytes(const mqc_t4 *d, int32_t dtype, int32_t groups) {
    if (check_extents("group_norm_workspace_bytes", d, dtype, groups, MQC_ACT_NONE) != MQC_OK || d->d0 == 0) return 0;
    return part_bytes(d, dtype) + static_cast<size_t>(round_up(int64_t(d->d0) * groups * 8, 256));
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
    const size_t need = mqc_group_norm_workspace_bytes(xd, dtype, groups);
    if ((st = check_workspace(name, workspace, workspace_bytes, need)) != MQC_OK) return st;
    GnParams P{};
    fill(P, xd, groups);
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
    const mqc_t4 *all[2] = {xd, yd};
    return run(name, P, vector_of(dtype, all, 2), dtype, false, static_cast<cudaStream_t>(stream));
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
    const size_t need = mqc_group_norm_workspace_bytes(xd, dtype, groups);
    if ((st = check_workspace(name, workspace, workspace_bytes, need)) != MQC_OK) return st;
    GnParams P{};
    fill(P, xd, groups);
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
    P.coef = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + part_bytes(xd, dtype));
    const mqc_t4 *all[3] = {xd, gd, gxd};
    return run(name, P, vector_of(dtype, all, 3), dtype, true, s);
}

}  // extern "C"
