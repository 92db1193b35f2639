// linear.cuh -- the matrix products of a linear layer on the tensor cores
// (tcgen05.mma kind::f16, bf16 or fp16 operands, fp32 accumulators in tensor
// memory) with bias, activation and residual in the epilogue, and the passes
// around them.
//
// One kernel body serves all products D[i][j] = sum_r A[i][r] B[j][r]:
//   forward     y  = x . w^T      A = x (tokens),   B = w (features), both stored r-innermost
//   or swapped  y^T = w . x^T     A = w (features), B = x (tokens): few tokens
//   gx = dz . w                   B = w stored j-innermost
//   gw = dz^T . x                 A and B stored i- / j-innermost
// An operand stored with its own index innermost goes to the tensor core as
// an MN-major tile (64 indices x 64 reduction steps per TMA box), without a
// transposed copy.
#pragma once

#include "common.cuh"
#include "dense.cuh"

namespace mqc {

constexpr int kLinRows = 128;        // rows of A per tile
constexpr int kLinBK = 64;           // reduction steps per stage: one 128-byte swizzle row
constexpr int kLinMaxStages = 8;
constexpr int kLinThreads = 192;     // warp 0 TMA, warp 1 MMA, warps 2-5 read the accumulators
constexpr uint64_t kLinTimeoutNs = 4000000000ull;

struct LinParams {
    CUtensorMap amap, bmap;
    CUtensorMap ymap, zmap;          // CTA pairs with 16-byte output rows: boxes of 32 x 32 elements
    int32_t I, J, R;                 // extents of A's rows, B's rows and the reduction
    int32_t a_mn, b_mn;              // operand stored with its own index innermost
    int32_t swap;                    // i is the feature and j the token (else i the token)
    int32_t bn;                      // rows of B per tile, a multiple of 16
    int32_t tiles_i, tiles, splits, stages;
    int32_t b_bytes;                 // bytes of B per stage
    uint32_t idesc;
    int32_t act;
    int32_t vec_out;                 // output (and residual) rows are whole 16-byte vectors
    const float *bias;               // per feature
    const void *res;
    void *y, *z;
    int64_t ldr, ldy, ldz;
};

// The sums of a layer's bias gradient: gb[n] = sum of `slabs` partial rows.
struct BiasGrad {
    const float *part;
    float *gb;
    int32_t slabs, N;
};

// One launch: one or two products (of the same tile width where CTA pairs run
// them) and a bias gradient's last sums.
struct LinGroup {
    LinParams p[2];
    int32_t first;                   // tiles (single tiles: clusters) of p[0]; those of p[1] follow
    int32_t tiles;                   // of both
    int32_t early, late_from;        // CTA pairs: see pair_tile
    int32_t cluster;                 // single tiles: CTAs of a cluster, a multiple of both products' splits
    BiasGrad bias;                   // gb NULL: none
};

// One column's partial rows, in row order over four running sums.
__device__ __forceinline__ void bias_grad_column(const BiasGrad &b, int c) {
    float s[4] = {};
    int k = 0;
    for (; k + 4 <= b.slabs; k += 4)
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] += b.part[static_cast<int64_t>(k + q) * b.N + c];
    for (; k < b.slabs; ++k) s[0] += b.part[static_cast<int64_t>(k) * b.N + c];
    b.gb[c] = (s[0] + s[1]) + (s[2] + s[3]);
}

// Instruction descriptor of kind::f16 with fp32 accumulators (bit 4): operand
// formats at bits 7 and 10 (0 = fp16, 1 = bf16), MN-major A at bit 15 and B at
// bit 16, N>>3 at 17..22, M>>4 at 24..28.
__host__ __device__ constexpr uint32_t make_idesc_f16(bool bf16, bool a_mn, bool b_mn, uint32_t M, uint32_t N) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
        "[%2];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
        : "memory");
}

// D[tmem] (+)= A[smem] . B[smem]^T, 16-bit operands of one type, K = 16.
__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    return a;
}
struct LinFew {
    const void *x, *w;
    const float *bias;
    const void *res;
    void *y, *z;
    int64_t ldx, ldw, ldr, ldy, ldz;
    int32_t M, N, K, act;
};

// bias, activation and residual of one element, z and y stored.
template <typename T, typename Params>
__device__ __forceinline__ void lin_store(const Params &P, float v, int64_t m, int n) {
    if (P.bias) v += __ldg(P.bias + n);
    if (P.z) static_cast<T *>(P.z)[m * P.ldz + n] = from_f32<T>(v);
    v = act_value(P.act, v);
    if (P.res) v += to_f32(static_cast<const T *>(P.res)[m * P.ldr + n]);
    static_cast<T *>(P.y)[m * P.ldy + n] = from_f32<T>(v);
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, float a, float b, float c, float d) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d)
                 : "memory");
}

// A CTA's share of a tile: `rows` tokens from m0 on, `width` features from n0
// on, summed from the SPLITS partial copies [rows_all][ld] in its shared memory
// in order, finished and stored, eight features a thread.  VEC: the rows are
// whole 16-byte vectors; else they are cut at the 16-byte boundaries of y, and
// the ends stored as single elements.  (Both gradients of 509 x 777 x 1003: one
// feature a lane 18.4 us, with a branch around each element's loads 20.5, now
// 14.1.)
template <typename T, int SPLITS, bool VEC>
__device__ __forceinline__ void tile_epilogue(const LinParams &P, const float *part, int ld, int rows_all, int rows,
                                              int width, int64_t m0, int n0) {
    const T *res = static_cast<const T *>(P.res);
    T *y = static_cast<T *>(P.y), *z = static_cast<T *>(P.z);
    if (VEC) {
        const int groups = width / 8;
        for (int e = threadIdx.x; e < rows * groups; e += kLinThreads) {
            const int o = e / groups, n = (e - o * groups) * 8;
            const int64_t m = m0 + o;
            uint4 r = make_uint4(0, 0, 0, 0);
            if (res) r = *reinterpret_cast<const uint4 *>(res + m * P.ldr + n0 + n);
            float v[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float4 s = *reinterpret_cast<const float4 *>(part + o * ld + n + 4 * h);
#pragma unroll
                for (int c = 1; c < SPLITS; ++c) {
                    const float4 t = *reinterpret_cast<const float4 *>(part + (c * rows_all + o) * ld + n + 4 * h);
                    s.x += t.x, s.y += t.y, s.z += t.z, s.w += t.w;
                }
                if (P.bias) {
                    const float4 b = __ldg(reinterpret_cast<const float4 *>(P.bias + n0 + n) + h);
                    s.x += b.x, s.y += b.y, s.z += b.z, s.w += b.w;
                }
                v[4 * h] = s.x, v[4 * h + 1] = s.y, v[4 * h + 2] = s.z, v[4 * h + 3] = s.w;
            }
            if (z) *reinterpret_cast<uint4 *>(z + m * P.ldz + n0 + n) = Vec<T>::narrow(v);
            act_values(P.act, v);
            if (res) {
                float f[8];
                Vec<T>::widen(r, f);
                add_to(v, f);
            }
            *reinterpret_cast<uint4 *>(y + m * P.ldy + n0 + n) = Vec<T>::narrow(v);
        }
        return;
    }
    const int across = (width + 14) / 8;   // the most runs of a row
    const bool z_alike = ((P.ldz ^ P.ldy) & 7) == 0, res_alike = ((P.ldr ^ P.ldy) & 7) == 0;
    for (int e = threadIdx.x; e < rows * across; e += kLinThreads) {
        const int o = e / across;
        const int64_t m = m0 + o;
        const int n = (e - o * across) * 8 - static_cast<int>((m * P.ldy + n0) & 7);
        if (n >= width) continue;
        const int lo = max(0, -n), hi = min(8, width - n);
        const bool whole = lo == 0 && hi == 8;
        T *to = y + m * P.ldy + n0 + n;
        // what lies outside reads its neighbour's: no branches between the loads
        float v[8], f[8] = {};
        int at[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) at[q] = min(max(n + q, 0), width - 1);
        if (res && whole && res_alike) {
            Vec<T>::widen(*reinterpret_cast<const uint4 *>(res + m * P.ldr + n0 + n), f);
        } else if (res) {
#pragma unroll
            for (int q = 0; q < 8; ++q) f[q] = to_f32(res[m * P.ldr + n0 + at[q]]);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = part[o * ld + at[q]];
#pragma unroll
        for (int c = 1; c < SPLITS; ++c)
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] += part[(c * rows_all + o) * ld + at[q]];
        if (P.bias) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] += __ldg(P.bias + n0 + at[q]);
        }
        if (z && whole && z_alike) {
            *reinterpret_cast<uint4 *>(z + m * P.ldz + n0 + n) = Vec<T>::narrow(v);
        } else if (z) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q >= lo && q < hi) z[m * P.ldz + n0 + n + q] = from_f32<T>(v[q]);
        }
        act_values(P.act, v);
        if (res) add_to(v, f);
        if (whole) {
            *reinterpret_cast<uint4 *>(to) = Vec<T>::narrow(v);
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q >= lo && q < hi) to[q] = from_f32<T>(v[q]);
        }
    }
}

// One 128 x bn tile of D for each `splits` CTAs of a cluster, which share its
// reduction (contiguous runs of 64-step blocks).  Once all of them are through
// with their stages, each sends the c-th part of its fp32 partial tile to the
// shared memory of the c-th (writes, which nobody waits for; reading the parts
// back from their owners spent most of a small product's time on the latency
// of distributed shared memory), and after another barrier every CTA sums what
// it got in rank order and stores it.  So a product with few tiles uses all
// SMs in one launch, without a workspace, and gives the same bits each time.
// Small products are bound by latency: a launch, the first stages, a barrier
// for the join, the epilogue.  128 x 1003 x 515 fp16 takes 9.6 us with the
// copies of both operands before it, where its 1.4 MB would take 0.2; both
// gradients of 509 x 777 x 1003 14.1 us with the copies and dz.
template <typename T>
__global__ void __launch_bounds__(kLinThreads) linear_tile_kernel(const __grid_constant__ LinGroup G) {
    extern __shared__ uint8_t lin_smem_raw[];
    __shared__ uint64_t full[kLinMaxStages], empty[kLinMaxStages], done;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    uint8_t *smem = lin_smem_raw + ((1024u - (smem_u32(lin_smem_raw) & 1023u)) & 1023u);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    int id = blockIdx.x / G.cluster;
    const int place = blockIdx.x - id * G.cluster;
    if (id >= G.tiles) {   // clusters behind the tiles': the bias gradient
        wait_previous();
        const int c = (blockIdx.x - G.tiles * G.cluster) * kLinThreads + threadIdx.x;
        if (c < G.bias.N) bias_grad_column(G.bias, c);
        return;
    }
    const LinParams &P = G.p[id >= G.first];
    if (id >= G.first) id -= G.first;
    const int sub = place / P.splits, rank = place - sub * P.splits;   // which of the cluster's tiles, whose part
    const int tile = id * (G.cluster / P.splits) + sub;
    if (tile >= P.tiles) {   // the last cluster's empty places keep its barriers
        cluster_sync();
        cluster_sync();
        return;
    }
    const int i0 = (tile % P.tiles_i) * kLinRows, j0 = (tile / P.tiles_i) * P.bn;
    const int nkb = (P.R + kLinBK - 1) / kLinBK;
    const int kb0 = static_cast<int>(static_cast<int64_t>(nkb) * rank / P.splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(nkb) * (rank + 1) / P.splits);
    const int a_bytes = kLinRows * kLinBK * 2;
    const int stage_bytes = a_bytes + P.b_bytes;
    const uint32_t tmem_cols = P.bn <= 32 ? 32 : P.bn <= 64 ? 64 : P.bn <= 128 ? 128 : 256;

    if (warp == 0) {
        if (lane == 0) {
            prefetch_tensormap(&P.amap);
            prefetch_tensormap(&P.bmap);
            for (int s = 0; s < P.stages; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], 1);
            }
            mbar_init(&done, 1);
            abort_flag = 0;
            fence_mbar_init();
        }
    } else if (warp == 1) {
        tmem_alloc(&tmem_base, tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_previous();
    asm volatile("fence.proxy.async.global;" ::: "memory");   // the copies are read by TMA
    const uint32_t tmem = tmem_base;
    volatile int *abort = &abort_flag;

    if (warp == 0) {
        const bool issuer = elect_one();
        int s = 0, ph = 0, issued = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (kb - kb0 >= P.stages && !mbar_wait(&empty[s], ph ^ 1, kLinTimeoutNs, abort)) break;
            if (issuer) {
                uint8_t *a = smem + s * stage_bytes, *b = a + a_bytes;
                mbar_arrive_expect_tx(&full[s], stage_bytes);
                if (P.a_mn) {
                    tma_load_2d(a, &P.amap, &full[s], i0 * 2, kb * kLinBK);
                    tma_load_2d(a + 8192, &P.amap, &full[s], (i0 + 64) * 2, kb * kLinBK);
                } else {
                    tma_load_2d(a, &P.amap, &full[s], kb * kLinBK * 2, i0);
                }
                if (P.b_mn) {
                    for (int j = 0; j < P.b_bytes / 8192; ++j)
                        tma_load_2d(b + j * 8192, &P.bmap, &full[s], (j0 + 64 * j) * 2, kb * kLinBK);
                } else {
                    tma_load_2d(b, &P.bmap, &full[s], kb * kLinBK * 2, j0);
                }
            }
            __syncwarp();
            ++issued;
            if (++s == P.stages) {
                s = 0;
                ph ^= 1;
            }
        }
        // a wait that ran out leaves copies in flight: let the last ones land
        // (bounded) before the shared memory is given up
        if (*abort)
            for (int k = 0; k < min(issued, P.stages); ++k) {
                const int n = issued - 1 - k;
                mbar_wait(&full[n % P.stages], (n / P.stages) & 1, 100000000ull, nullptr);
            }
    } else if (warp == 1) {
        const bool issuer = elect_one();
        const uint32_t a_step = P.a_mn ? 2048 : 32, b_step = P.b_mn ? 2048 : 32;
        int s = 0, ph = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1 && ok; ++kb) {
            ok = mbar_wait(&full[s], ph, kLinTimeoutNs, abort);
            if (!ok) break;
            tc_fence_after();
            if (issuer) {
                const uint32_t a = smem_u32(smem + s * stage_bytes), b = a + a_bytes;
#pragma unroll
                for (int k = 0; k < kLinBK / 16; ++k) {
                    // K-major: 8-row groups 1024 bytes apart.  MN-major: 8-step
                    // groups 1024 bytes apart, the next 64 indices 8192 bytes on.
                    const uint64_t ad = make_smem_desc(a + k * a_step, P.a_mn ? 8192 : 16, 1024, kSwizzle128B);
                    const uint64_t bd = make_smem_desc(b + k * b_step, P.b_mn ? 8192 : 16, 1024, kSwizzle128B);
                    tc_mma_f16(tmem, ad, bd, P.idesc, (kb > kb0 || k > 0) ? 1u : 0u);
                }
                tc_commit(&empty[s]);
            }
            __syncwarp();
            if (++s == P.stages) {
                s = 0;
                ph ^= 1;
            }
        }
        if (issuer) tc_commit(&done);
        __syncwarp();
    }

    // partial tile -> [outer][inner], the output's row index (token) outer: i
    // outer in the plain form, j outer in the swapped one; the CTA of rank c
    // gets rows [c, c + 1) * share of all partial tiles, [rank][share][ld]
    float *part = reinterpret_cast<float *>(smem);
    const int outer = P.swap ? P.bn : kLinRows, share = outer / P.splits;
    const int ld = P.swap ? kLinRows : P.bn + 4;   // 16-byte rows, and lanes' vectors in distinct banks
    if (warp >= 2) {
        mbar_wait(&done, 0, kLinTimeoutNs, abort);
        tc_fence_after();
    }
    __syncthreads();
    if (G.cluster > 1) cluster_sync();   // nobody's stages are in use any more
    if (warp >= 2) {
        const int quad = warp & 3, i = quad * 32 + lane;
        const uint32_t base = smem_u32(part);
        const int mine = i / share;      // plain form: the CTA that gets row i
        const uint32_t row = P.swap ? 0 : map_to_rank(base, sub * P.splits + mine) +
                                              4 * ((rank * share + i - mine * share) * ld);
        for (int c = 0; c < P.bn; c += 16) {
            uint32_t r[16];
            tc_ld_32x32b_x16(tmem + (static_cast<uint32_t>(quad * 32) << 16) + c, r);
            tc_wait_ld();
            if (P.swap) {
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const int o = c + q, owner = o / share;
                    st_cluster_f32(map_to_rank(base, sub * P.splits + owner) +
                                       4 * ((rank * share + o - owner * share) * ld + i),
                                   __uint_as_float(r[q]));
                }
            } else {
#pragma unroll
                for (int q = 0; q < 16; q += 4)
                    st_cluster_v4(row + 4 * (c + q), __uint_as_float(r[q]), __uint_as_float(r[q + 1]),
                                  __uint_as_float(r[q + 2]), __uint_as_float(r[q + 3]));
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (G.cluster > 1) cluster_sync();   // all parts have arrived
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, tmem_cols);
    }

    const int inner = P.swap ? kLinRows : P.bn;
    const int64_t m0 = (P.swap ? j0 : i0) + rank * share;
    const int n0 = P.swap ? i0 : j0;
    const int M = P.swap ? P.J : P.I, N = P.swap ? P.I : P.J;
    const int rows = static_cast<int>(min(static_cast<int64_t>(share), M - m0)), width = min(inner, N - n0);
    if (P.vec_out) {
        if (P.splits == 1) tile_epilogue<T, 1, true>(P, part, ld, share, rows, width, m0, n0);
        else if (P.splits == 2) tile_epilogue<T, 2, true>(P, part, ld, share, rows, width, m0, n0);
        else if (P.splits == 4) tile_epilogue<T, 4, true>(P, part, ld, share, rows, width, m0, n0);
        else tile_epilogue<T, 8, true>(P, part, ld, share, rows, width, m0, n0);
    } else {
        if (P.splits == 1) tile_epilogue<T, 1, false>(P, part, ld, share, rows, width, m0, n0);
        else if (P.splits == 2) tile_epilogue<T, 2, false>(P, part, ld, share, rows, width, m0, n0);
        else if (P.splits == 4) tile_epilogue<T, 4, false>(P, part, ld, share, rows, width, m0, n0);
        else tile_epilogue<T, 8, false>(P, part, ld, share, rows, width, m0, n0);
    }
}

// ---------------------------------------------------------------- CTA pairs
// TMA load into this CTA's shared memory that completes on a barrier of either
// CTA of the pair (`bar`: shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void tc_mma_f16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// One arrival on the barrier at this offset in both CTAs of the pair, when the
// MMAs issued so far have completed.
__device__ __forceinline__ void tc_commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

constexpr int kPairThreads = 320;    // warp 0 TMA, warp 1 MMA, warps 2-9 the epilogue
constexpr int kPairMaxStages = 8;

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
                 "r"(src), "r"(c0), "r"(c1)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

constexpr int kPairBuf = 2048;       // one 32 x 32 block of 16-bit outputs
constexpr int kPairStaging = 8 * 2 * kPairBuf;

// The epilogue of one warp: 32 tokens (one a lane) x 32 features.  A lane
// stores its 64 bytes of y (and z) to a shared-memory block in the 64-byte
// swizzle of the output's tensor map, which the TMA writes out as whole
// sectors, clipped at the matrix's ends (whole 16 bytes of a row only, which
// is why matrices of other widths take the other form).  (Stores of 16 bytes a lane straight
// to global memory, rows apart, were half sectors: with z they cost 40 us of
// 221 at 8192 x 4096 x 4096.)
template <typename T>
struct PairEpilogue {
    const LinParams &P;
    uint8_t *buf;                    // two blocks
    int lane, &turn;
    __device__ PairEpilogue(const LinParams &p, uint8_t *b, int l, int &t) : P(p), buf(b), lane(l), turn(t) {}

    __device__ __forceinline__ void send(const CUtensorMap *map, const float (&v)[32], int m, int n) {
        uint8_t *dst = buf + turn * kPairBuf;
        turn ^= 1;
        // this block's last copy has been read (the other one's may be running)
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float e[8] = {v[8 * q],     v[8 * q + 1], v[8 * q + 2], v[8 * q + 3],
                                v[8 * q + 4], v[8 * q + 5], v[8 * q + 6], v[8 * q + 7]};
            *reinterpret_cast<uint4 *>(dst + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) = Vec<T>::narrow(e);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tma_store_2d(map, smem_u32(dst), n * 2, m);
        __syncwarp();
    }

    // The lane's 64 bytes of the residual (its rows are whole 16-byte vectors).
    __device__ __forceinline__ void fetch(uint4 (&r)[4], int64_t m, int n) const {
        const T *res = static_cast<const T *>(P.res) + m * P.ldr + n;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            r[q] = m < P.I && n + 8 * q < P.J ? reinterpret_cast<const uint4 *>(res)[q] : make_uint4(0, 0, 0, 0);
    }

    __device__ __forceinline__ void block(const uint32_t (&acc)[32], const uint4 (&r)[4], int m0, int n) {
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(acc[e]);
        if (P.bias) {
            if (n + 32 <= P.J) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float4 b = __ldg(reinterpret_cast<const float4 *>(P.bias + n) + q);
                    v[4 * q] += b.x, v[4 * q + 1] += b.y, v[4 * q + 2] += b.z, v[4 * q + 3] += b.w;
                }
            } else {
                const float b = n + lane < P.J ? __ldg(P.bias + n + lane) : 0.f;
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] += __shfl_sync(0xFFFFFFFFu, b, e);
            }
        }
        if (P.z) send(&P.zmap, v, m0, n);
        act_values(P.act, v);
        if (P.res) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float f[8];
                Vec<T>::widen(r[q], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * q + e] += f[e];
            }
        }
        send(&P.ymap, v, m0, n);
    }

    // Output rows of other strides: the accumulators change lanes through
    // shared memory (fp32; a row's elements in an order exclusive-ored with its
    // number, so that neither side meets bank conflicts), and a warp writes 32
    // features of one token at a time.  (64 features in 4-byte words took
    // longer: the odd rows' ends need stores of their own.)
    __device__ __forceinline__ void block_any(const uint32_t (&acc)[32], float bias, int64_t m0, int n) {
        float *f = reinterpret_cast<float *>(buf);
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 32; ++e) f[lane * 32 + (e ^ lane)] = __uint_as_float(acc[e]);
        __syncwarp();
        if (n + lane >= P.J) return;
        const int rows = static_cast<int>(min(static_cast<int64_t>(32), P.I - m0));
        const T *res = P.res ? static_cast<const T *>(P.res) + m0 * P.ldr + n + lane : nullptr;
        T *y = static_cast<T *>(P.y) + m0 * P.ldy + n + lane;
        T *z = P.z ? static_cast<T *>(P.z) + m0 * P.ldz + n + lane : nullptr;
        const int64_t ldy = P.ldy, ldz = P.ldz, ldr = P.ldr;
        const int act = P.act;
        constexpr int U = 8;   // rows whose operands are in flight together
        for (int e = 0; e < rows; e += U) {
            float v[U], r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                v[u] = f[(e + u) * 32 + (lane ^ (e + u))] + bias;
                r[u] = res && e + u < rows ? to_f32(res[u * ldr]) : 0.f;
            }
            if (z) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (e + u < rows) z[u * ldz] = from_f32<T>(v[u]);
                z += U * ldz;
            }
            act_values(act, v);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (e + u < rows) y[u * ldy] = from_f32<T>(res ? v[u] + r[u] : v[u]);
            y += U * ldy;
            if (res) res += U * ldr;
        }
    }
};

// The n-th tile of pair c of `pairs`, or -1.  The tiles of the first product
// (the longer reduction) are dealt out in turn.  Pairs from `late_from` on got
// one of them less; they take `early` tiles of the second product in its
// stead, and the rest of those is dealt out in turn again.  (8192 x 2048 x
// 2048: 64 tiles of 128 blocks, then 256 of 32 on 74 pairs; dealt out in turn
// alone the busiest pair has 256 blocks, so 224.)
__device__ __forceinline__ int pair_tile(const LinGroup &G, int c, int pairs, int n) {
    const int own = G.first > c ? (G.first - c - 1) / pairs + 1 : 0;
    if (n < own) return c + n * pairs;
    n -= own;
    int at = G.first;
    if (G.early > 0) {
        const int late = pairs - G.late_from;
        if (c >= G.late_from) {
            if (n < G.early) return at + (c - G.late_from) + n * late;
            n -= G.early;
        }
        at += G.early * late;
    }
    at += c + n * pairs;
    return at < G.tiles ? at : -1;
}

// Large products: a persistent pair of CTAs (one per SM) computes 256 x bn
// tiles with tcgen05.mma.cta_group::2.  Each CTA holds 128 rows of A and half
// of B's rows per stage, so an SM reads half the operand bytes from shared
// memory per product that a lone CTA would; its tensor memory holds two
// accumulators of 128 x bn, so that the epilogue of one tile runs beside the
// products of the next.  All full-stage signals go to the first CTA, which
// issues the products for both.
// Bound by the tensor cores: 8192 x 4096 x 4096 bf16 with bias, GELU, residual
// and z stored takes 205 us, 1340 TFLOP/s (78% of a library product's rate in
// a burst, 92% of its rate under the power limit), the tensor pipe active for
// 83% of it; both gradients of 8192 x 2048 x 2048 with dz and the bias' sums
// before them 117 us.  (Tiles of lone CTAs: 306 and 170 us.)
template <typename T>
__global__ void __launch_bounds__(kPairThreads, 1) linear_pair_kernel(const __grid_constant__ LinGroup G) {
    extern __shared__ uint8_t lin_smem_raw[];
    __shared__ uint64_t full[kPairMaxStages], empty[kPairMaxStages], acc_full[2], acc_empty[2];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    uint8_t *smem = lin_smem_raw + ((1024u - (smem_u32(lin_smem_raw) & 1023u)) & 1023u);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank();
    const int a_bytes = kLinRows * kLinBK * 2;
    // the same for both products
    const int bn = G.p[0].bn, b_bytes = G.p[0].b_bytes, stages = G.p[0].stages;
    const int stage_bytes = a_bytes + b_bytes;
    const int pairs = gridDim.x / 2, me = blockIdx.x / 2;
    volatile int *abort = &abort_flag;

    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&G.p[0].amap);
        prefetch_tensormap(&G.p[0].bmap);
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 16);   // eight epilogue warps of each CTA
        }
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    wait_previous();
    asm volatile("fence.proxy.async.global;" ::: "memory");   // the copies are read by TMA
    const uint32_t tmem = tmem_base;

    // tile t: bands of eight rows of tiles, column by column inside a band,
    // so that the tiles in flight share their operands in L2
    auto place = [&](int t, int &i0, int &j0) -> const LinParams & {
        const LinParams &P = G.p[t >= G.first];
        if (t >= G.first) t -= G.first;
        const int tiles_j = (P.J + bn - 1) / bn;
        const int band = t / (8 * tiles_j), in = t - band * 8 * tiles_j;
        const int rows = min(8, P.tiles_i - band * 8);
        i0 = (band * 8 + in % rows) * 2 * kLinRows;
        j0 = (in / rows) * bn;
        return P;
    };

    if (warp == 0) {
        const bool issuer = elect_one();
        int s = 0, ph = 0, issued = 0;
        bool ok = true;
        for (int n = 0, t; ok && (t = pair_tile(G, me, pairs, n)) >= 0; ++n) {
            int i0, j0;
            const LinParams &P = place(t, i0, j0);
            const int nkb = (P.R + kLinBK - 1) / kLinBK;
            i0 += rank * kLinRows;
            j0 += rank * (bn / 2);
            for (int kb = 0; kb < nkb; ++kb) {
                if (issued >= stages && !mbar_wait(&empty[s], ph ^ 1, kLinTimeoutNs, abort)) {
                    ok = false;
                    break;
                }
                if (issuer) {
                    uint8_t *a = smem + s * stage_bytes, *b = a + a_bytes;
                    const uint32_t bar = map_to_rank(smem_u32(&full[s]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * stage_bytes);
                    if (P.a_mn) {
                        tma_load_2d_pair(a, &P.amap, bar, i0 * 2, kb * kLinBK);
                        tma_load_2d_pair(a + 8192, &P.amap, bar, (i0 + 64) * 2, kb * kLinBK);
                    } else {
                        tma_load_2d_pair(a, &P.amap, bar, kb * kLinBK * 2, i0);
                    }
                    if (P.b_mn) {
                        for (int j = 0; j < b_bytes / 8192; ++j)
                            tma_load_2d_pair(b + j * 8192, &P.bmap, bar, (j0 + 64 * j) * 2, kb * kLinBK);
                    } else {
                        tma_load_2d_pair(b, &P.bmap, bar, kb * kLinBK * 2, j0);
                    }
                }
                __syncwarp();
                ++issued;
                if (++s == stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        // the last copies land before the shared memory is given up: their
        // stages are consumed (empty) in the normal course, and given time to
        // land after a wait that ran out
        for (int k = 0; k < min(issued, stages); ++k) {
            const int n = issued - 1 - k;
            mbar_wait(&empty[n % stages], (n / stages) & 1, *abort ? 100000000ull : kLinTimeoutNs, nullptr);
        }
    } else if (warp == 1 && rank == 0) {
        const bool issuer = elect_one();
        int s = 0, ph = 0;
        bool ok = true;
        for (int n = 0, t; ok && (t = pair_tile(G, me, pairs, n)) >= 0; ++n) {
            const LinParams &P = G.p[t >= G.first];
            const int nkb = (P.R + kLinBK - 1) / kLinBK;
            const uint32_t a_step = P.a_mn ? 2048 : 32, b_step = P.b_mn ? 2048 : 32;
            const uint32_t a_lbo = P.a_mn ? 8192 : 16, b_lbo = P.b_mn ? 8192 : 16, idesc = P.idesc;
            const int b = n & 1;
            if (n >= 2 && !mbar_wait(&acc_empty[b], ((n >> 1) & 1) ^ 1, kLinTimeoutNs, abort)) break;
            tc_fence_after();
            for (int kb = 0; kb < nkb; ++kb) {
                if (!mbar_wait(&full[s], ph, kLinTimeoutNs, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (issuer) {
                    const uint32_t a = smem_u32(smem + s * stage_bytes), bs = a + a_bytes;
#pragma unroll
                    for (int k = 0; k < kLinBK / 16; ++k) {
                        const uint64_t ad = make_smem_desc(a + k * a_step, a_lbo, 1024, kSwizzle128B);
                        const uint64_t bd = make_smem_desc(bs + k * b_step, b_lbo, 1024, kSwizzle128B);
                        tc_mma_f16_pair(tmem + b * bn, ad, bd, idesc, (kb > 0 || k > 0) ? 1u : 0u);
                    }
                    tc_commit_pair(&empty[s]);
                }
                __syncwarp();
                if (++s == stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
            if (issuer && ok) tc_commit_pair(&acc_full[b]);
            __syncwarp();
        }
    } else if (warp == 1) {
        // the second CTA's: the bias gradient
        if (G.bias.gb)
            for (int c = me * 32 + lane; c < G.bias.N; c += pairs * 32) bias_grad_column(G.bias, c);
    } else {
        // warps 2-9: a quadrant of the rows, half of the columns
        const int quad = warp & 3, half = (warp - 2) / 4;
        int turn = 0;
        for (int n = 0, t; (t = pair_tile(G, me, pairs, n)) >= 0; ++n) {
            const int b = n & 1;
            int i0, j0;
            const LinParams &P = place(t, i0, j0);
            PairEpilogue<T> out(P, smem + stages * stage_bytes + (warp - 2) * 2 * kPairBuf, lane, turn);
            i0 += rank * kLinRows + quad * 32;
            j0 += half * (bn / 2);
            uint4 r[4];
            if (P.res && P.vec_out) out.fetch(r, i0 + lane, j0);
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&acc_full[b], (n >> 1) & 1, kLinTimeoutNs, abort))) break;
            tc_fence_after();
            for (int c = 0; c < bn / 2; c += 32) {
                const int mine = j0 + c + lane;   // block_any's column, asked for before the accumulators
                const float bias = !P.vec_out && P.bias && mine < P.J ? __ldg(P.bias + mine) : 0.f;
                uint32_t acc[32];
                tc_ld_32x32b_x32(tmem + (static_cast<uint32_t>(quad * 32) << 16) + b * bn + half * (bn / 2) + c,
                                 acc);
                tc_wait_ld();
                const bool last = c + 32 == bn / 2;
                if (last) {   // read in full: the accumulator may be overwritten
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(&acc_empty[b]), 0));
                }
                if (i0 >= P.I || j0 + c >= P.J) continue;
                if (P.vec_out) {
                    uint4 now[4] = {r[0], r[1], r[2], r[3]};
                    if (P.res && !last) out.fetch(r, i0 + lane, j0 + c + 32);
                    out.block(acc, now, i0, j0 + c);
                } else {
                    out.block_any(acc, bias, i0, j0 + c);
                }
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// ---------------------------------------------------------------- few tokens
// One to eight tokens: the weights are read once, and that is all there is.
// A block of eight warps computes RN features; the warps share the reduction
// in chunks of 256 steps, a lane 8 of them from 16-byte loads (VEC), and are
// joined in warp order.  Nothing but the loads' latency stands between the
// launch and the last byte: 1 x 4096 x 4096 takes 8.5 us, 3.9 TB/s (a plain
// copy of 6.45 TB/s would read the weights in 5.2; its 1024 blocks find 592
// places, so that a second, partial round starts with cold loads); the
// tensor-core form spends more on filling its pipeline and joining its CTAs
// (11.4 us).  At 1 x 8192 x 8192, 5.3 TB/s.
template <typename T, int MT, int RN, bool VEC>
__global__ void __launch_bounds__(256) linear_few_kernel(const LinFew P) {
    __shared__ float sums[8][RN * MT];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int n0 = blockIdx.x * RN;
    const T *w = static_cast<const T *>(P.w) + static_cast<int64_t>(n0) * P.ldw, *x = static_cast<const T *>(P.x);
    float2 acc[RN][MT];
#pragma unroll
    for (int r = 0; r < RN; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[r][m] = make_float2(0.f, 0.f);
    const int chunks = (P.K + 255) / 256;
#pragma unroll 1   // 62 registers, four blocks an SM; two steps at once gain nothing
    for (int c = warp; c < chunks; c += 8) {
        const int k = c * 256 + (VEC ? lane * 8 : lane);
        float wv[RN][8];
        if (VEC && k + 8 <= P.K) {
            uint4 raw[RN];
#pragma unroll
            for (int r = 0; r < RN; ++r)
                raw[r] = n0 + r < P.N ? __ldcs(reinterpret_cast<const uint4 *>(w + r * P.ldw + k)) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < RN; ++r) Vec<T>::widen(raw[r], wv[r]);
        } else {
            const int stride = VEC ? 1 : 32;
#pragma unroll
            for (int r = 0; r < RN; ++r)
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    wv[r][q] = n0 + r < P.N && k + q * stride < P.K ? to_f32(w[r * P.ldw + k + q * stride]) : 0.f;
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float xv[8];
            if (m >= P.M) continue;
            if (VEC && k + 8 <= P.K) {
                Vec<T>::widen(__ldg(reinterpret_cast<const uint4 *>(x + m * P.ldx + k)), xv);
            } else {
                const int stride = VEC ? 1 : 32;
#pragma unroll
                for (int q = 0; q < 8; ++q) xv[q] = k + q * stride < P.K ? to_f32(x[m * P.ldx + k + q * stride]) : 0.f;
            }
#pragma unroll
            for (int r = 0; r < RN; ++r)
#pragma unroll
                for (int q = 0; q < 8; q += 2)
                    acc[r][m] = fma2(make_float2(wv[r][q], wv[r][q + 1]), make_float2(xv[q], xv[q + 1]), acc[r][m]);
        }
    }
    // sums over the lanes: at each step a lane keeps half of the values and
    // sends the other half away, then the one value that is left goes round
    constexpr int V = RN * MT;
    float v[V];
#pragma unroll
    for (int r = 0; r < RN; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) v[m * RN + r] = acc[r][m].x + acc[r][m].y;
    int index = 0;
#pragma unroll
    for (int half = V / 2, o = 16; half > 0; half /= 2, o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float got = __shfl_xor_sync(0xFFFFFFFFu, up ? v[i] : v[i + half], o);
            v[i] = (up ? v[i + half] : v[i]) + got;
        }
        index += up ? half : 0;
    }
#pragma unroll
    for (int o = 16 / V; o > 0; o /= 2) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
    if ((lane & (32 / V - 1)) == 0) sums[warp][index] = v[0];
    __syncthreads();
    if (threadIdx.x < RN * MT) {
        const int m = threadIdx.x / RN, n = n0 + threadIdx.x % RN;
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) v += sums[k][threadIdx.x];
        if (m < P.M && n < P.N) lin_store<T>(P, v, m, n);
    }
}

// ---------------------------------------------------------------- passes before the products
// Copy of a matrix whose rows are not multiples of 16 bytes into rows of
// round_up(cols, 8) elements (the tensor maps' stride rule).
struct PackJob {
    const uint16_t *src;
    uint16_t *dst;
    int64_t ld, rows, ldd;
    int32_t cols, blocks;
};
__device__ __forceinline__ void pack_rows(const PackJob &J, int block) {
    const int64_t per = J.ldd / 8, n = J.rows * per;
    for (int64_t e = block * 256ll + threadIdx.x; e < n; e += J.blocks * 256ll) {
        const int64_t r = n <= 0x7FFFFFFF ? static_cast<uint32_t>(e) / static_cast<uint32_t>(per) : e / per;
        const int c0 = static_cast<int>(e - r * per) * 8;
        const uint16_t *src = J.src + r * J.ld + c0;
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (c0 + q < J.cols) w[q / 2] |= static_cast<uint32_t>(src[q]) << (16 * (q & 1));
        *reinterpret_cast<uint4 *>(J.dst + r * J.ldd + c0) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// dz = g * act'(z) (rounded to the operand type of the products) and the
// column sums of the unrounded dz over a slab of rows.  A block is 32 lanes x
// 8 row groups; a lane owns 8 columns.  VEC: whole 16-byte loads.  Bound by
// memory: 8192 x 2048 bf16 with z (100 MB) takes 17 us, 5.9 TB/s.
constexpr int kDzRows = 8;
struct DzJob {
    const void *g, *z;               // z NULL: dz = g
    void *dz;                        // NULL: sums only
    float *part;                     // [slabs][N], NULL: no sums
    int64_t ldg, ldz, lddz;
    int32_t M, N, act, slab, col_blocks, blocks;
};
template <typename T, bool VEC>
__device__ __forceinline__ void dz_block(const DzJob &J, int block) {
    __shared__ float sums[kDzRows][32][9];
    const T *g = static_cast<const T *>(J.g), *z = static_cast<const T *>(J.z);
    T *dz = static_cast<T *>(J.dz);
    const int by = block / J.col_blocks, bx = block - by * J.col_blocks;
    const int lane = threadIdx.x % 32, ty = threadIdx.x / 32;
    const int c0 = (bx * 32 + lane) * 8;
    const int r1 = static_cast<int>(min(static_cast<int64_t>(J.M), (by + static_cast<int64_t>(1)) * J.slab));
    float acc[8] = {};
    auto finish = [&](float (&v)[8], const float (&zv)[8], int64_t r) {
        if (z) {
            float s[8];
            act_slopes(J.act, zv, s);
            mul_to(v, s);
        }
        add_to(acc, v);
        if (dz) *reinterpret_cast<uint4 *>(dz + r * J.lddz + c0) = Vec<T>::narrow(v);   // lddz = round_up(N, 8)
    };
    int64_t r = static_cast<int64_t>(by) * J.slab + ty;
    if (VEC && c0 + 8 <= J.N) {
        // the next two rows are under way while two are worked on
        constexpr int U = 2;
        const T *gp = g + r * J.ldg + c0, *zp = z ? z + r * J.ldz + c0 : nullptr;
        const int64_t gs = kDzRows * J.ldg, zs = kDzRows * J.ldz;
        uint4 gr[U] = {}, zr[U] = {}, gn[U] = {}, zn[U] = {};
        auto load = [&](uint4 (&a)[U], uint4 (&b)[U], int64_t row) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (row + u * kDzRows < r1) {
                    a[u] = *reinterpret_cast<const uint4 *>(gp + u * gs);
                    if (z) b[u] = *reinterpret_cast<const uint4 *>(zp + u * zs);
                }
            gp += U * gs;
            if (z) zp += U * zs;
        };
        load(gr, zr, r);
#pragma unroll 2
        for (; r < r1; r += U * kDzRows) {
            load(gn, zn, r + U * kDzRows);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r + u * kDzRows < r1) {
                    float v[8], zv[8];
                    Vec<T>::widen(gr[u], v);
                    Vec<T>::widen(zr[u], zv);
                    finish(v, zv, r + u * kDzRows);
                }
                gr[u] = gn[u];
                zr[u] = zn[u];
            }
        }
    } else if (c0 < J.N) {
        for (; r < r1; r += kDzRows) {
            float v[8], zv[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                v[q] = c0 + q < J.N ? to_f32(g[r * J.ldg + c0 + q]) : 0.f;
                zv[q] = z && c0 + q < J.N ? to_f32(z[r * J.ldz + c0 + q]) : 0.f;
            }
            finish(v, zv, r);
        }
    }
    if (J.part == nullptr) return;
#pragma unroll
    for (int q = 0; q < 8; ++q) sums[ty][lane][q] = acc[q];
    __syncthreads();
    // 256 columns of the block, one per thread
    const int l = threadIdx.x / 8, q = threadIdx.x % 8, c = (bx * 32 + l) * 8 + q;
    if (c < J.N) {
        float s = 0.f;
        for (int k = 0; k < kDzRows; ++k) s += sums[k][l][q];
        J.part[static_cast<int64_t>(by) * J.N + c] = s;
    }
}

// All that has to be done before a layer's products, in one launch: the dz
// blocks, then those of up to two copies.
struct LinPrep {
    DzJob dz;
    PackJob pack[2];
    int64_t blocks() const { return int64_t(dz.blocks) + pack[0].blocks + pack[1].blocks; }
};
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, 3) linear_prep_kernel(const __grid_constant__ LinPrep P) {
    let_next_start();
    int b = blockIdx.x;
    if (b < P.dz.blocks) return dz_block<T, VEC>(P.dz, b);
    b -= P.dz.blocks;
    const int which = b >= P.pack[0].blocks;
    pack_rows(P.pack[which], which ? b - P.pack[0].blocks : b);
}

static __global__ void linear_bias_grad_kernel(const BiasGrad b) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c < b.N) bias_grad_column(b, c);
}

}  // namespace mqc
