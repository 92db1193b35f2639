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
struct Product {
    Operand X, W;
    int32_t tokens, features, red;
    Epilogue E;
    // few tokens: the features fill the 128 rows of the tensor core's tile
    // and the tokens its columns, so that no rows are spent on padding
    bool swap() const { return tokens <= 64; }
    int64_t kblocks() const { return ceil_div(red, kLinBK); }
};

// Whether the rows of the outputs and the residual are whole 16-byte vectors
// (a TMA store clips its rows at whole 16 bytes only).
bool vector_rows(const Product &p) {
    const Epilogue &E = p.E;
    return p.features % 8 == 0 && E.ldy % 8 == 0 && (!E.z || E.ldz % 8 == 0) && (!E.res || E.ldr % 8 == 0);
}

// What both kernels need besides the tiling.
mqc_status fill_params(LinParams &P, const Product &p, bool bf16, int rows, bool pair) {
    const Operand &A = P.swap ? p.W : p.X, &B = P.swap ? p.X : p.W;
    const Epilogue &E = p.E;
    P.R = p.red;
    P.a_mn = A.mn;
    P.b_mn = B.mn;
    P.idesc = make_idesc_f16(bf16, A.mn, B.mn, rows, P.bn);
    P.vec_out = vector_rows(p);
    P.act = E.act;
    P.bias = E.bias;
    P.res = E.res;
    P.y = E.y;
    P.z = E.z;
    P.ldr = E.ldr;
    P.ldy = E.ldy;
    P.ldz = E.ldz;
    mqc_status st = A.mn ? encode_matrix_map(&P.amap, A.p, p.red, P.I, A.ld, kLinBK)
                         : encode_matrix_map(&P.amap, A.p, P.I, p.red, A.ld, kLinRows);
    if (st != MQC_OK) return st;
    st = B.mn ? encode_matrix_map(&P.bmap, B.p, p.red, P.J, B.ld, kLinBK)
              : encode_matrix_map(&P.bmap, B.p, P.J, p.red, B.ld, pair ? P.bn / 2 : P.bn);
    if (st == MQC_OK && pair && P.vec_out) st = encode_matrix_map(&P.ymap, E.y, P.I, P.J, E.ldy, 32, 64);
    if (st == MQC_OK && pair && P.vec_out && E.z) st = encode_matrix_map(&P.zmap, E.z, P.I, P.J, E.ldz, 32, 64);
    return st;
}

mqc_status launch_group(const LinGroup &G, bool pair, bool bf16, int64_t grid, int cluster, int threads, int smem,
                        bool after, const DeviceLimits &d, cudaStream_t stream) {
    if (grid > (int64_t(1) << 31) - 1) return fail(MQC_ERR_INVALID, "linear: too many tiles");
    void (*kernel)(LinGroup) = pair ? (bf16 ? linear_pair_kernel<__nv_bfloat16> : linear_pair_kernel<__half>)
                                    : (bf16 ? linear_tile_kernel<__nv_bfloat16> : linear_tile_kernel<__half>);
    mqc_status st = allow_smem(reinterpret_cast<const void *>(kernel), 2 * pair + bf16, d);
    if (st != MQC_OK) return st;
    const Launch launch(grid, threads, cluster, smem, after, stream);
    cudaError_t e = cudaLaunchKernelEx(&launch.cfg, kernel, G);
    return e == cudaSuccess ? MQC_OK : cuda_fail(e, "linear kernel launch");
}

// The tiling of a product on single tiles, and its estimated time in us, from
// a fit to some 300 measured combinations on a B200 (within 20%): 4.4 for a
// launch, 2.7 for a joined reduction, 3.8 for each further round of resident
// CTAs, and for each CTA of the busiest SM 0.16 a stage of 64 steps plus 0.27
// by its columns (of 256), and 6.3 by its columns to finish them (16 where the
// output's rows are not whole vectors).  Clusters of
// four and eight CTAs, an SM each, find room for fewer (in whole groups of
// SMs).
struct TilePlan {
    int32_t bn, splits;
    int64_t tiles;
    double us;
};
TilePlan plan_tiles(const Product &p, int sms) {
    const bool swap = p.swap(), vec = vector_rows(p);
    const int64_t rows = ceil_div(swap ? p.features : p.tokens, kLinRows), cols = swap ? p.tokens : p.features;
    TilePlan best{0, 0, 0, 1e300};
    for (int bn = 256; bn >= 32; bn /= 2) {
        TilePlan t{bn, 1, 0, 0.0};
        if (swap) {   // all the tokens in one tile, so that the weights are read once
            t.bn = static_cast<int32_t>(round_up(cols, 16));
            bn = 32;
        } else if (bn > 32 && bn / 2 >= cols) {
            continue;
        }
        t.tiles = rows * ceil_div(cols, t.bn);
        for (t.splits = 1; t.splits <= 8 && t.splits <= p.kblocks(); t.splits *= 2) {
            const int64_t room = t.splits == 8 ? sms * 13 / 16 : (t.splits == 4 ? sms * 9 / 10 : sms);
            const int64_t on_sm = ceil_div(t.tiles * t.splits, room), kb = ceil_div(p.kblocks(), t.splits);
            const int64_t rounds = t.bn <= 64 ? ceil_div(on_sm, 2) : on_sm;   // two narrow tiles share an SM
            const double wide = t.bn / 256.0;
            t.us = 4.4 + (t.splits > 1 ? 2.7 : 0.0) + (rounds - 1) * 3.8 +
                   on_sm * (kb * (0.16 + 0.27 * wide) + (vec ? 6.3 : 16.0) * wide / t.splits);
            if (t.us < best.us) best = t;
        }
    }
    return best;
}

// On CTA pairs: the launch at 5.6, and for the busiest pair either its 64-step
// blocks at 0.40 (256 columns) or 0.32 and the last tile's output, or all of
// its tiles' outputs after the first one's blocks, whichever takes longer.  A
// tile's output takes 4.7 or 2.8, 10.4 or 6.2 where the rows are not whole
// vectors.
struct PairPlan {
    int32_t bn;
    double us;
};
int64_t pair_tiles(const Product &p, int bn) { return ceil_div(p.tokens, 2 * kLinRows) * ceil_div(p.features, bn); }
// How the second product's tiles make up for the first's last, partial round
// (pair_tile): as many as weigh one of the first's, for each pair without one.
void deal(int64_t t0, int64_t t1, int64_t kb0, int64_t kb1, int pairs, int32_t &early, int32_t &late_from) {
    late_from = static_cast<int32_t>(t0 % pairs);
    early = 0;
    if (t1 > 0 && late_from > 0)
        early = static_cast<int32_t>(std::min((kb0 + kb1 / 2) / kb1, t1 / (pairs - late_from)));
}
PairPlan plan_pairs(const Product *const *p, int count, int pairs) {
    PairPlan best{0, 1e300};
    for (int bn = 256; bn >= 128; bn /= 2) {
        const int64_t t0 = pair_tiles(*p[0], bn), t1 = count > 1 ? pair_tiles(*p[1], bn) : 0;
        const int64_t kb0 = p[0]->kblocks(), kb1 = count > 1 ? p[1]->kblocks() : 1;
        int32_t early, late_from;
        deal(t0, t1, kb0, kb1, pairs, early, late_from);
        const double block = bn == 256 ? 0.40 : 0.32;
        const auto output = [bn](const Product &p) { return vector_rows(p) ? 0.9 + bn / 68.0 : 2.0 + bn / 30.5; };
        const double e0 = output(*p[0]), e1 = count > 1 ? output(*p[1]) : e0;
        double us = 0.0;
        const int64_t rest = t1 - int64_t(early) * (pairs - late_from);
        const int64_t each0 = t0 / pairs, each1 = rest / pairs, more1 = rest % pairs;
        for (int64_t c : {int64_t(0), int64_t(late_from), more1}) {   // where the pairs' shares change
            const int64_t n0 = each0 + (c < late_from), n1 = each1 + (c < more1) + (c >= late_from ? early : 0);
            us = std::max({us, (n0 * kb0 + n1 * kb1) * block + e1, n0 * e0 + n1 * e1 + kb0 * block});
        }
        us += 5.6;
        if (us < best.us) best = PairPlan{bn, us};
    }
    return best;
}

// One or two products on CTA pairs, the longer reduction's tiles first (they
// are dealt out in turn, and the shorter ones even out the end).
mqc_status launch_pairs(const Product *p, int count, const BiasGrad &bias, bool bf16, bool after,
                        const DeviceLimits &d, cudaStream_t stream) {
    const int pairs = d.sms / 2;
    const Product *order[2] = {&p[0], count > 1 ? &p[1] : nullptr};
    if (count > 1 && p[1].kblocks() > p[0].kblocks()) std::swap(order[0], order[1]);
    const int bn = plan_pairs(order, count, pairs).bn;
    const int b_bytes = bn / 2 * kLinBK * 2, stage = kLinRows * kLinBK * 2 + b_bytes;
    LinGroup G{};
    const int stages = std::min(kPairMaxStages, (d.max_smem - 2048 - 1024 - kPairStaging) / stage);
    G.bias = bias;
    int64_t tiles = 0;
    for (int i = 0; i < count; ++i) {
        LinParams &P = G.p[i];
        P.I = order[i]->tokens;
        P.J = order[i]->features;
        P.bn = bn;
        P.b_bytes = b_bytes;
        P.stages = stages;
        P.splits = 1;
        P.tiles_i = static_cast<int32_t>(ceil_div(P.I, 2 * kLinRows));
        tiles += pair_tiles(*order[i], bn);
        if (tiles > (int64_t(1) << 30)) return fail(MQC_ERR_INVALID, "linear: too many tiles");
        if (i == 0) G.first = static_cast<int32_t>(tiles);
        mqc_status st = fill_params(P, *order[i], bf16, 2 * kLinRows, true);
        if (st != MQC_OK) return st;
    }
    G.tiles = static_cast<int32_t>(tiles);
    if (count > 1 && tiles >= pairs)
        deal(G.first, tiles - G.first, order[0]->kblocks(), order[1]->kblocks(), pairs, G.early, G.late_from);
    return launch_group(G, true, bf16, 2 * std::min<int64_t>(tiles, pairs), 2, kPairThreads,
                        1024 + stages * stage + kPairStaging, after, d, stream);
}

// One or two products on single tiles.  A product's plan does not depend on
// the other's presence, nor then do its bits.
// The room for a CTA's part of a tile also keeps the CTAs that fit on an SM to
// its 512 columns of tensor memory together (at worst eight with 64 for 48
// tokens, in 25.6 KB each), so that no cluster waits for
// columns which another, waiting one holds.
mqc_status launch_tiles(const Product *p, int count, const BiasGrad &bias, bool bf16, bool after,
                        const DeviceLimits &d, cudaStream_t stream) {
    LinGroup G{};
    G.bias = bias;
    G.cluster = 1;
    int64_t ctas = 0;
    for (int i = 0; i < count; ++i) {
        LinParams &P = G.p[i];
        P.swap = p[i].swap();
        P.I = P.swap ? p[i].features : p[i].tokens;
        P.J = P.swap ? p[i].tokens : p[i].features;
        P.tiles_i = static_cast<int32_t>(ceil_div(P.I, kLinRows));
        const TilePlan t = plan_tiles(p[i], d.sms);
        if (t.tiles > (int64_t(1) << 30) / 16) return fail(MQC_ERR_INVALID, "linear: too many tiles");
        P.bn = t.bn;
        P.tiles = static_cast<int32_t>(t.tiles);
        P.splits = t.splits;
        G.cluster = std::max(G.cluster, P.splits);
        ctas += t.tiles * P.splits;
    }
    int smem = 0;
    for (int i = 0; i < count; ++i) {
        LinParams &P = G.p[i];
        const bool b_mn = P.swap ? p[i].X.mn : p[i].W.mn;
        P.b_bytes = (b_mn ? static_cast<int>(round_up(P.bn, 64)) : P.bn) * kLinBK * 2;
        const int stage = kLinRows * kLinBK * 2 + P.b_bytes;
        const int part = P.swap ? P.bn * kLinRows * 4 : kLinRows * (P.bn + 4) * 4;
        const int room = d.max_smem - 2048 - 1024;
        const int share = ctas > d.sms && P.bn <= 64 ? room / 2 - 512 : room;
        P.stages = std::max(1, std::min({kLinMaxStages, share / stage,
                                         static_cast<int>(ceil_div(p[i].kblocks(), P.splits))}));
        smem = std::max(smem, 1024 + std::max(P.stages * stage, part));
        G.tiles += static_cast<int32_t>(ceil_div(P.tiles, G.cluster / P.splits));   // clusters
        if (i == 0) G.first = G.tiles;
        mqc_status st = fill_params(P, p[i], bf16, kLinRows, false);
        if (st != MQC_OK) return st;
    }
    const int64_t extra = bias.gb ? round_up(ceil_div(bias.N, kLinThreads), G.cluster) : 0;
    return launch_group(G, false, bf16, int64_t(G.tiles) * G.cluster + extra, G.cluster, kLinThreads, smem, after, d,
                        stream);
}

// The products of a call, and its bias gradient's last sums beside them: in
// one launch when the same kernel suits them.  after: linear_prep_kernel runs
// before them.
mqc_status launch_products(const Product *p, int count, const BiasGrad &bias, int32_t dtype, bool after,
                           const DeviceLimits &d, cudaStream_t stream) {
    const bool bf16 = dtype == MQC_BF16;
    bool pairs[2] = {};
    for (int i = 0; i < count; ++i) {
        const Product *one = &p[i];
        pairs[i] = !one->swap() && plan_pairs(&one, 1, d.sms / 2).us < plan_tiles(*one, d.sms).us;
    }
    if (count > 1 && pairs[0] != pairs[1]) {
        mqc_status st = launch_products(p, 1, bias, dtype, after, d, stream);
        return st != MQC_OK ? st : launch_products(p + 1, 1, BiasGrad{}, dtype, false, d, stream);
    }
    return pairs[0] ? launch_pairs(p, count, bias, bf16, after, d, stream)
                    : launch_tiles(p, count, bias, bf16, after, d, stream);
}

// Bytes of a padded copy of a rows x cols matrix, and whether one is needed.
bool needs_pack(int64_t ld) { return ld % 8 != 0; }
size_t packed_bytes(int64_t rows, int64_t cols) {
    return static_cast<size_t>(round_up(rows * round_up(cols, 8) * 2, 256));
}

// Plans the copy of an operand, if its rows need one, into the workspace at ws.
void plan_pack(PackJob &job, Operand &op, int64_t rows, int64_t cols, uint8_t *&ws, const DeviceLimits &d) {
    if (!needs_pack(op.ld)) return;
    job.src = static_cast<const uint16_t *>(op.p);
    job.dst = reinterpret_cast<uint16_t *>(ws);
    job.ld = op.ld;
    job.rows = rows;
    job.cols = static_cast<int32_t>(cols);
    job.ldd = round_up(cols, 8);
    job.blocks = static_cast<int32_t>(std::min<int64_t>(ceil_div(rows * (job.ldd / 8), 256), int64_t(d.sms) * 8));
    op.p = ws;
    op.ld = job.ldd;
    ws += packed_bytes(rows, cols);
}

mqc_status launch_prep(const LinPrep &prep, int32_t dtype, cudaStream_t stream) {
    const int64_t blocks = prep.blocks();
    if (blocks == 0) return MQC_OK;
    if (blocks > (int64_t(1) << 31) - 1) return fail(MQC_ERR_INVALID, "linear: too many blocks");
    const bool vec = prep.dz.ldg % 8 == 0 && (prep.dz.z == nullptr || prep.dz.ldz % 8 == 0);
    const unsigned grid = static_cast<unsigned>(blocks);
    if (dtype == MQC_BF16) {
        if (vec) linear_prep_kernel<__nv_bfloat16, true><<<grid, 256, 0, stream>>>(prep);
        else linear_prep_kernel<__nv_bfloat16, false><<<grid, 256, 0, stream>>>(prep);
    } else {
        if (vec) linear_prep_kernel<__half, true><<<grid, 256, 0, stream>>>(prep);
        else linear_prep_kernel<__half, false><<<grid, 256, 0, stream>>>(prep);
    }
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MQC_OK : cuda_fail(e, "linear_prep_kernel launch");
}

// One to eight tokens (linear_few_kernel).  Four features a block where that
// still leaves several blocks an SM, else one.
// One token always, a few where the weights are few; at N x K this form against
// the tensor cores', in us:
//   tokens        1            2            4            6            8
//   1024 x 1024    2.7,  6.2    2.9,  6.3    5.2,  6.3    6.0,  6.3    6.7,  6.5
//   2048 x 2048    3.4,  7.8    5.1,  7.9    6.1,  7.9    7.2,  7.9    8.0,  7.9
//   4096 x 4096    8.6, 11.9   11.5, 11.8   17.1, 12.1   20.2, 12.1
//   8192 x 8192   25.7, 29.2   30.9, 28.6   47.5, 28.7
// (where those would have to copy operands first, two and eight).
bool few_tokens(const mqc_linear *l) {
    const bool copies = needs_pack(l->ldx) || needs_pack(l->ldw);
    const int64_t weights = int64_t(l->N) * l->K;
    if (l->M <= 2) return l->M == 1 || copies || weights <= int64_t(1) << 24;
    return weights <= int64_t(1) << 22 && l->M <= (copies ? 8 : 6);
}
template <typename T, int MT, int RN>
void launch_few_as(const LinFew &P, bool vec, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(ceil_div(P.N, RN));
    if (vec) linear_few_kernel<T, MT, RN, true><<<grid, 256, 0, s>>>(P);
    else linear_few_kernel<T, MT, RN, false><<<grid, 256, 0, s>>>(P);
}
template <typename T>
void launch_few(const LinFew &P, cudaStream_t s) {
    const bool vec = P.ldw % 8 == 0 && (P.M == 1 || P.ldx % 8 == 0), wide = P.N >= 2048;
    if (P.M == 1) wide ? launch_few_as<T, 1, 4>(P, vec, s) : launch_few_as<T, 1, 1>(P, vec, s);
    else if (P.M == 2) wide ? launch_few_as<T, 2, 4>(P, vec, s) : launch_few_as<T, 2, 1>(P, vec, s);
    else if (P.M <= 4) wide ? launch_few_as<T, 4, 4>(P, vec, s) : launch_few_as<T, 4, 1>(P, vec, s);
    else wide ? launch_few_as<T, 8, 4>(P, vec, s) : launch_few_as<T, 8, 1>(P, vec, s);
}

mqc_status check_linear(const mqc_linear *l, const char *name) {
    if (l == nullptr) return fail(MQC_ERR_INVALID, "%s: null descriptor", name);
    if (l->M < 0 || l->N <= 0 || l->K <= 0) return fail(MQC_ERR_INVALID, "%s: bad extents", name);
    // row numbers and byte offsets in a row stay within 31 bits
    if (l->M > (1 << 30) || l->N > (1 << 29) || l->K > (1 << 29))
        return fail(MQC_ERR_INVALID, "%s: M above 2^30, or N or K above 2^29", name);
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

// Row slabs of the dz pass: all blocks (three on each of 148 SMs) at once, at
// least 32 rows each.  A function of the sizes alone, so that the workspace
// query needs no device.
void dz_slabs(int64_t M, int64_t N, int32_t &slab, int32_t &slabs) {
    const int64_t col_blocks = ceil_div(N, 256);
    const int64_t want = std::max<int64_t>(1, 148 * 3 / col_blocks);
    slab = static_cast<int32_t>(std::max<int64_t>(32, ceil_div(M, want)));
    slabs = static_cast<int32_t>(ceil_div(M, slab));
}

}  // namespace
}  // namespace mqc

using namespace mqc;

extern "C" {

size_t mqc_linear_fwd_workspace_bytes(const mqc_linear *l) {
    if (check_linear(l, "linear_fwd") != MQC_OK || few_tokens(l)) return 0;
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
    if (few_tokens(l)) {
        LinFew P{x, w, bias, residual, y, z, l->ldx, l->ldw, l->ldr, l->ldy, l->ldz, l->M, l->N, l->K, l->act};
        if (l->dtype == MQC_BF16) launch_few<__nv_bfloat16>(P, s);
        else launch_few<__half>(P, s);
        cudaError_t e = cudaGetLastError();
        return e == cudaSuccess ? MQC_OK : cuda_fail(e, "linear_few_kernel launch");
    }
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    Product p{{x, l->ldx, false}, {w, l->ldw, false}, l->M, l->N, l->K, {}};
    LinPrep prep{};
    plan_pack(prep.pack[0], p.X, l->M, l->K, ws, d);
    plan_pack(prep.pack[1], p.W, l->N, l->K, ws, d);
    if ((st = launch_prep(prep, l->dtype, s)) != MQC_OK) return st;
    p.E.bias = bias;
    p.E.res = residual;
    p.E.y = y;
    p.E.z = z;
    p.E.ldr = l->ldr;
    p.E.ldy = l->ldy;
    p.E.ldz = l->ldz;
    p.E.act = l->act;
    return launch_products(&p, 1, BiasGrad{}, l->dtype, prep.blocks() > 0, d, s);
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
    BiasGrad bias{gb ? reinterpret_cast<float *>(ws) : nullptr, gb, slabs, l->N};
    ws += round_up(int64_t(slabs) * l->N * 4, 256);
    LinPrep prep{};
    Operand DZ{g, l->ldg, false};
    const bool copy = act || needs_pack(l->ldg);   // dz is not g as it stands
    if (gb || copy) {
        DzJob &J = prep.dz;
        J.g = g;
        J.z = act ? z : nullptr;
        J.part = gb ? reinterpret_cast<float *>(workspace) : nullptr;
        J.ldg = l->ldg;
        J.ldz = l->ldz;
        J.lddz = round_up(l->N, 8);
        J.M = l->M;
        J.N = l->N;
        J.act = l->act;
        J.slab = slab;
        J.col_blocks = static_cast<int32_t>(ceil_div(l->N, 256));
        if (int64_t(J.col_blocks) * slabs > (int64_t(1) << 30)) return fail(MQC_ERR_INVALID, "%s: too many blocks", name);
        J.blocks = J.col_blocks * slabs;
        if (copy && (gx || gw)) {
            J.dz = ws;
            DZ.p = ws;
            DZ.ld = J.lddz;
        }
        if (copy) ws += packed_bytes(l->M, l->N);
    }
    Product p[2];
    int count = 0;
    if (gx) {
        p[count] = Product{DZ, {w, l->ldw, true}, l->M, l->K, l->N, {}};
        plan_pack(prep.pack[0], p[count].W, l->N, l->K, ws, d);
        p[count].E.y = gx;
        p[count++].E.ldy = l->ldgx;
    }
    if (gw) {
        Operand G = DZ;
        G.mn = true;
        p[count] = Product{G, {x, l->ldx, true}, l->N, l->K, l->M, {}};
        plan_pack(prep.pack[1], p[count].W, l->M, l->K, ws, d);
        p[count].E.y = gw;
        p[count++].E.ldy = l->ldgw;
    }
    if ((st = launch_prep(prep, l->dtype, s)) != MQC_OK) return st;
    if (count > 0) return launch_products(p, count, bias, l->dtype, prep.blocks() > 0, d, s);
    linear_bias_grad_kernel<<<static_cast<unsigned>(ceil_div(l->N, 128)), 128, 0, s>>>(bias);
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MQC_OK : cuda_fail(e, "linear_bias_grad_kernel launch");
}

}  // extern "C"
