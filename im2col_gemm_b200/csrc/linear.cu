// linear.cu -- entry points of the linear layer (include/mqc.h): argument
// checks, the choice of the product's tiles, and the launches of linear.cuh.
#include "linear.cuh"

#include <algorithm>
#include <atomic>

#include "host.h"

namespace mqc {

cudaError_t linear_take_device_error(int *value) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(value, g_mqc_device_error, sizeof *value);
    if (e == cudaSuccess && *value != 0) e = cudaMemcpyToSymbol(g_mqc_device_error, &zero, sizeof zero);
    return e;
}

namespace {

// A product's operand: index i (or j) by reduction step.  mn: stored with the
// index innermost ([reduction][index]), else [index][reduction].
struct Operand {
    const void *p;
    int64_t ld;
    bool mn;
};

struct Epilogue {
    const float *bias = nullptr;
    const void *res = nullptr;
    void *y = nullptr, *z = nullptr;
    int64_t ldr = 0, ldy = 0, ldz = 0;
    int act = MQC_ACT_NONE;
};

// Dynamic shared memory of a kernel, allowed once per device.
mqc_status allow_smem(const void *kernel, int index, const DeviceLimits &d) {
    static std::atomic<bool> done[4][64];
    if (done[index][d.device].load(std::memory_order_acquire)) return MQC_OK;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, d.max_smem - 2048);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(linear kernel)");
    done[index][d.device].store(true, std::memory_order_release);
    return MQC_OK;
}

// D[token][feature] = sum over `red` of X . W: X indexed by token, W by
// feature; the epilogue stores rows of tokens.
mqc_status launch_product(Operand X, Operand W, int32_t tokens, int32_t features, int32_t red, int32_t dtype,
                          const Epilogue &E, const DeviceLimits &d, cudaStream_t stream) {
    LinParams P;
    const bool bf16 = dtype == MQC_BF16;
    // few tokens: the features fill the 128 rows of the tensor core's tile
    // and the tokens its columns, so that no rows are spent on padding
    P.swap = tokens <= 64;
    const Operand &A = P.swap ? W : X, &B = P.swap ? X : W;
    P.I = P.swap ? features : tokens;
    P.J = P.swap ? tokens : features;
    P.R = red;
    P.a_mn = A.mn;
    P.b_mn = B.mn;
    P.splits = 1;
    const int nkb = static_cast<int>(ceil_div(red, kLinBK));
    const int room = d.max_smem - 2048 - 1024;
    int64_t grid;
    int cluster, threads, smem, a_rows, b_rows;
    // CTA pairs once their 256-row tiles fill most of the SM pairs
    const int64_t pair_rows = ceil_div(P.I, 2 * kLinRows);
    const int pairs = d.sms / 2;
    const bool pair = !P.swap && pair_rows * ceil_div(P.J, 128) >= pairs * 3 / 4;
    if (pair) {
        // 256 or 128 columns: the fewer rounds of tiles, a narrow tile counted
        // as 0.6 of a wide one
        const int64_t wide = ceil_div(pair_rows * ceil_div(P.J, 256), pairs) * 10;
        const int64_t narrow = ceil_div(pair_rows * ceil_div(P.J, 128), pairs) * 6;
        P.bn = narrow < wide ? 128 : 256;
        P.tiles_i = static_cast<int32_t>(pair_rows);
        P.b_bytes = P.bn / 2 * kLinBK * 2;
        const int64_t tiles = pair_rows * ceil_div(P.J, P.bn);
        const int stage = kLinRows * kLinBK * 2 + P.b_bytes;
        P.stages = std::min(kPairMaxStages, (room - kPairStaging) / stage);
        smem = 1024 + P.stages * stage + kPairStaging;
        grid = 2 * std::min<int64_t>(tiles, pairs);
        if (tiles > (int64_t(1) << 30)) return fail(MQC_ERR_INVALID, "linear: too many tiles");
        P.idesc = make_idesc_f16(bf16, P.a_mn, P.b_mn, 2 * kLinRows, P.bn);
        cluster = 2;
        threads = kPairThreads;
        a_rows = kLinRows;
        b_rows = P.bn / 2;
    } else {
        P.tiles_i = static_cast<int32_t>(ceil_div(P.I, kLinRows));
        // the widest column tile that still gives every SM one; all the tokens
        // of the swapped form in one tile, so that the weights are read once
        if (P.swap) {
            P.bn = static_cast<int32_t>(round_up(P.J, 16));
        } else {
            P.bn = 256;
            while (P.bn > 32 && (P.bn / 2 >= P.J || P.tiles_i * ceil_div(P.J, P.bn) < d.sms)) P.bn /= 2;
        }
        const int64_t tiles = P.tiles_i * ceil_div(P.J, P.bn);
        while (P.splits < 8 && tiles * P.splits < d.sms && nkb / (2 * P.splits) >= 2) P.splits *= 2;
        P.b_bytes = (P.b_mn ? static_cast<int>(round_up(P.bn, 64)) : P.bn) * kLinBK * 2;
        const int stage = kLinRows * kLinBK * 2 + P.b_bytes;
        const int part = P.swap ? P.bn * kLinRows * 4 : kLinRows * (P.bn + 1) * 4;
        const int share = tiles * P.splits > d.sms && P.bn <= 64 ? room / 2 - 512 : room;
        P.stages = std::max(1, std::min({kLinMaxStages, share / stage, static_cast<int>(ceil_div(nkb, P.splits))}));
        smem = 1024 + std::max(P.stages * stage, part);
        grid = tiles * P.splits;
        if (grid > (int64_t(1) << 31) - 1) return fail(MQC_ERR_INVALID, "linear: too many tiles");
        P.idesc = make_idesc_f16(bf16, P.a_mn, P.b_mn, kLinRows, P.bn);
        cluster = P.splits;
        threads = kLinThreads;
        a_rows = kLinRows;
        b_rows = P.bn;
    }
    P.tma_out = pair && E.ldy % 8 == 0 && (!E.z || E.ldz % 8 == 0) && (!E.res || E.ldr % 8 == 0);
    P.act = E.act;
    P.bias = E.bias;
    P.res = E.res;
    P.y = E.y;
    P.z = E.z;
    P.ldr = E.ldr;
    P.ldy = E.ldy;
    P.ldz = E.ldz;
    mqc_status st = A.mn ? encode_matrix_map(&P.amap, A.p, red, P.I, A.ld, kLinBK)
                         : encode_matrix_map(&P.amap, A.p, P.I, red, A.ld, a_rows);
    if (st != MQC_OK) return st;
    st = B.mn ? encode_matrix_map(&P.bmap, B.p, red, P.J, B.ld, kLinBK)
              : encode_matrix_map(&P.bmap, B.p, P.J, red, B.ld, b_rows);
    if (st != MQC_OK) return st;
    if (P.tma_out) {
        st = encode_matrix_map(&P.ymap, E.y, P.I, P.J, E.ldy, 32, 64);
        if (st == MQC_OK && E.z) st = encode_matrix_map(&P.zmap, E.z, P.I, P.J, E.ldz, 32, 64);
        if (st != MQC_OK) return st;
    }
    void (*kernel)(LinParams) = pair ? (bf16 ? linear_pair_kernel<__nv_bfloat16> : linear_pair_kernel<__half>)
                                     : (bf16 ? linear_tile_kernel<__nv_bfloat16> : linear_tile_kernel<__half>);
    if ((st = allow_smem(reinterpret_cast<const void *>(kernel), 2 * pair + bf16, d)) != MQC_OK) return st;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P);
    return e == cudaSuccess ? MQC_OK : cuda_fail(e, "linear kernel launch");
}

// Bytes of a padded copy of a rows x cols matrix, and whether one is needed.
bool needs_pack(int64_t ld) { return ld % 8 != 0; }
size_t packed_bytes(int64_t rows, int64_t cols) {
    return static_cast<size_t>(round_up(rows * round_up(cols, 8) * 2, 256));
}

mqc_status pack(Operand &op, int64_t rows, int64_t cols, uint8_t *&ws, cudaStream_t stream, const DeviceLimits &d) {
    if (!needs_pack(op.ld)) return MQC_OK;
    const int64_t ldd = round_up(cols, 8);
    const int64_t blocks = std::min<int64_t>(ceil_div(rows * (ldd / 8), 256), int64_t(d.sms) * 8);
    linear_pack_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
        static_cast<const uint16_t *>(op.p), op.ld, rows, static_cast<int32_t>(cols), reinterpret_cast<uint16_t *>(ws),
        ldd);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "linear_pack_kernel launch");
    op.p = ws;
    op.ld = ldd;
    ws += packed_bytes(rows, cols);
    return MQC_OK;
}

mqc_status check_linear(const mqc_linear *l, const char *name) {
    if (l == nullptr) return fail(MQC_ERR_INVALID, "%s: null descriptor", name);
    if (l->M < 0 || l->N <= 0 || l->K <= 0) return fail(MQC_ERR_INVALID, "%s: bad extents", name);
    if (!act_ok(l->act)) return fail(MQC_ERR_INVALID, "%s: bad activation", name);
    if (l->dtype == MQC_F32)
        return fail(MQC_ERR_UNSUPPORTED, "%s: fp32 operands (the tensor cores take bf16 or fp16)", name);
    if (l->dtype != MQC_BF16 && l->dtype != MQC_F16) return fail(MQC_ERR_INVALID, "%s: bad dtype", name);
    return MQC_OK;
}

// A matrix argument: present, 16-byte aligned, rows that do not overlap.
mqc_status check_matrix(const char *name, const char *what, const void *p, int64_t ld, int64_t cols) {
    if (p == nullptr) return fail(MQC_ERR_INVALID, "%s: %s is null", name, what);
    if (!aligned16(p)) return fail(MQC_ERR_ALIGNMENT, "%s: %s not 16-byte aligned", name, what);
    if (ld < cols || ld > (int64_t(1) << 38))
        return fail(MQC_ERR_INVALID, "%s: row stride of %s out of range", name, what);
    return MQC_OK;
}

mqc_status check_workspace(const char *name, const void *ws, size_t bytes, size_t need) {
    if (need == 0) return MQC_OK;
    if (ws == nullptr || bytes < need)
        return fail(MQC_ERR_WORKSPACE, "%s: needs %zu workspace bytes, got %zu", name, need, ws ? bytes : size_t(0));
    if (!aligned16(ws)) return fail(MQC_ERR_ALIGNMENT, "%s: workspace not 16-byte aligned", name);
    return MQC_OK;
}

// Row slabs of the dz pass: enough blocks for two waves of 8 blocks an SM, at
// least 32 rows each.  A function of the sizes alone, so that the workspace
// query needs no device.
void dz_slabs(int64_t M, int64_t N, int32_t &slab, int32_t &slabs) {
    const int64_t col_blocks = ceil_div(N, 256);
    const int64_t want = std::max<int64_t>(1, 1184 / col_blocks);
    slab = static_cast<int32_t>(std::max<int64_t>(32, ceil_div(M, want)));
    slabs = static_cast<int32_t>(ceil_div(M, slab));
}

template <typename T>
void launch_dz(const mqc_linear *l, const void *g, const void *z, void *dz, float *part, int32_t slab, int32_t slabs,
               cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(ceil_div(l->N, 256)), static_cast<unsigned>(slabs));
    const T *gp = static_cast<const T *>(g), *zp = static_cast<const T *>(z);
    const int64_t lddz = round_up(l->N, 8);
    if (l->ldg % 8 == 0 && (z == nullptr || l->ldz % 8 == 0))
        linear_dz_kernel<T, true><<<grid, 256, 0, stream>>>(gp, l->ldg, zp, l->ldz, l->M, l->N, l->act,
                                                            static_cast<T *>(dz), lddz, part, slab);
    else
        linear_dz_kernel<T, false><<<grid, 256, 0, stream>>>(gp, l->ldg, zp, l->ldz, l->M, l->N, l->act,
                                                             static_cast<T *>(dz), lddz, part, slab);
}

}  // namespace
}  // namespace mqc

using namespace mqc;

extern "C" {

size_t mqc_linear_fwd_workspace_bytes(const mqc_linear *l) {
    if (check_linear(l, "linear_fwd") != MQC_OK) return 0;
    return (needs_pack(l->ldx) ? packed_bytes(l->M, l->K) : 0) + (needs_pack(l->ldw) ? packed_bytes(l->N, l->K) : 0);
}

mqc_status mqc_linear_fwd(const mqc_linear *l, const void *x, const void *w, const float *bias, const void *residual,
                          void *y, void *z, void *workspace, size_t workspace_bytes, void *stream) {
    const char *name = "linear_fwd";
    mqc_status st = check_linear(l, name);
    if (st != MQC_OK) return st;
    if (l->M == 0) return MQC_OK;
    if ((st = check_matrix(name, "x", x, l->ldx, l->K)) != MQC_OK) return st;
    if ((st = check_matrix(name, "w", w, l->ldw, l->K)) != MQC_OK) return st;
    if ((st = check_matrix(name, "y", y, l->ldy, l->N)) != MQC_OK) return st;
    if (residual && (st = check_matrix(name, "residual", residual, l->ldr, l->N)) != MQC_OK) return st;
    if (z && (st = check_matrix(name, "z", z, l->ldz, l->N)) != MQC_OK) return st;
    if (bias && !aligned16(bias)) return fail(MQC_ERR_ALIGNMENT, "%s: bias not 16-byte aligned", name);
    if ((st = check_workspace(name, workspace, workspace_bytes, mqc_linear_fwd_workspace_bytes(l))) != MQC_OK)
        return st;
    DeviceLimits d;
    if ((st = device_limits(&d)) != MQC_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    Operand X{x, l->ldx, false}, W{w, l->ldw, false};
    if ((st = pack(X, l->M, l->K, ws, s, d)) != MQC_OK) return st;
    if ((st = pack(W, l->N, l->K, ws, s, d)) != MQC_OK) return st;
    Epilogue E;
    E.bias = bias;
    E.res = residual;
    E.y = y;
    E.z = z;
    E.ldr = l->ldr;
    E.ldy = l->ldy;
    E.ldz = l->ldz;
    E.act = l->act;
    return launch_product(X, W, l->M, l->N, l->K, l->dtype, E, d, s);
}

size_t mqc_linear_bwd_workspace_bytes(const mqc_linear *l) {
    if (check_linear(l, "linear_bwd") != MQC_OK || l->M == 0) return 0;
    int32_t slab, slabs;
    dz_slabs(l->M, l->N, slab, slabs);
    size_t n = static_cast<size_t>(round_up(int64_t(slabs) * l->N * 4, 256));
    if (l->act != MQC_ACT_NONE || needs_pack(l->ldg)) n += packed_bytes(l->M, l->N);
    if (needs_pack(l->ldx)) n += packed_bytes(l->M, l->K);
    if (needs_pack(l->ldw)) n += packed_bytes(l->N, l->K);
    return n;
}

mqc_status mqc_linear_bwd(const mqc_linear *l, const void *g, const void *z, const void *x, const void *w, void *gx,
                          void *gw, float *gb, void *workspace, size_t workspace_bytes, void *stream) {
    const char *name = "linear_bwd";
    mqc_status st = check_linear(l, name);
    if (st != MQC_OK) return st;
    if (gw && (st = check_matrix(name, "gw", gw, l->ldgw, l->K)) != MQC_OK) return st;
    if (gb && !aligned16(gb)) return fail(MQC_ERR_ALIGNMENT, "%s: gb not 16-byte aligned", name);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (l->M == 0) {
        cudaError_t e = cudaSuccess;
        if (gw) e = cudaMemset2DAsync(gw, l->ldgw * 2, 0, size_t(l->K) * 2, l->N, s);
        if (e == cudaSuccess && gb) e = cudaMemsetAsync(gb, 0, size_t(l->N) * 4, s);
        return e == cudaSuccess ? MQC_OK : cuda_fail(e, "linear_bwd memset");
    }
    const bool act = l->act != MQC_ACT_NONE;
    if ((st = check_matrix(name, "g", g, l->ldg, l->N)) != MQC_OK) return st;
    if (act && (st = check_matrix(name, "z", z, l->ldz, l->N)) != MQC_OK) return st;
    if (gx && (st = check_matrix(name, "gx", gx, l->ldgx, l->K)) != MQC_OK) return st;
    if (gx && (st = check_matrix(name, "w", w, l->ldw, l->K)) != MQC_OK) return st;
    if (gw && (st = check_matrix(name, "x", x, l->ldx, l->K)) != MQC_OK) return st;
    if ((st = check_workspace(name, workspace, workspace_bytes, mqc_linear_bwd_workspace_bytes(l))) != MQC_OK)
        return st;
    if (!gx && !gw && !gb) return MQC_OK;
    DeviceLimits d;
    if ((st = device_limits(&d)) != MQC_OK) return st;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    int32_t slab, slabs;
    dz_slabs(l->M, l->N, slab, slabs);
    float *part = gb ? reinterpret_cast<float *>(ws) : nullptr;
    ws += round_up(int64_t(slabs) * l->N * 4, 256);
    Operand DZ{g, l->ldg, false};
    void *dz = nullptr;
    if ((gx || gw) && (act || needs_pack(l->ldg))) {
        dz = ws;
        DZ.p = dz;
        DZ.ld = round_up(l->N, 8);
    }
    if (act || needs_pack(l->ldg)) ws += packed_bytes(l->M, l->N);
    if (dz || part) {
        if (l->dtype == MQC_BF16) launch_dz<__nv_bfloat16>(l, g, act ? z : nullptr, dz, part, slab, slabs, s);
        else launch_dz<__half>(l, g, act ? z : nullptr, dz, part, slab, slabs, s);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_fail(e, "linear_dz_kernel launch");
    }
    if (part) {
        linear_bias_grad_kernel<<<static_cast<unsigned>(ceil_div(l->N, 128)), 128, 0, s>>>(part, slabs, l->N, gb);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_fail(e, "linear_bias_grad_kernel launch");
    }
    if (gx) {
        Operand W{w, l->ldw, true};
        if ((st = pack(W, l->N, l->K, ws, s, d)) != MQC_OK) return st;
        Epilogue E;
        E.y = gx;
        E.ldy = l->ldgx;
        if ((st = launch_product(DZ, W, l->M, l->K, l->N, l->dtype, E, d, s)) != MQC_OK) return st;
    }
    if (gw) {
        Operand X{x, l->ldx, true};
        if ((st = pack(X, l->M, l->K, ws, s, d)) != MQC_OK) return st;
        Operand G = DZ;
        G.mn = true;
        Epilogue E;
        E.y = gw;
        E.ldy = l->ldgw;
        if ((st = launch_product(G, X, l->N, l->K, l->M, l->dtype, E, d, s)) != MQC_OK) return st;
    }
    return MQC_OK;
}

}  // extern "C"
