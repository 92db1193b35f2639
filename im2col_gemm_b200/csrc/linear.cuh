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
    int32_t I, J, R;                 // extents of A's rows, B's rows and the reduction
    int32_t a_mn, b_mn;              // operand stored with its own index innermost
    int32_t swap;                    // i is the feature and j the token (else i the token)
    int32_t bn;                      // rows of B per tile, a multiple of 16
    int32_t tiles_i, splits, stages;
    int32_t b_bytes;                 // bytes of B per stage
    uint32_t idesc;
    int32_t act;
    const float *bias;               // per feature
    const void *res;
    void *y, *z;
    int64_t ldr, ldy, ldz;
};

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
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    return a;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// bias, activation and residual of one element, z and y stored.
template <typename T>
__device__ __forceinline__ void lin_store(const LinParams &P, float v, int64_t m, int n) {
    if (P.bias) v += __ldg(P.bias + n);
    if (P.z) static_cast<T *>(P.z)[m * P.ldz + n] = from_f32<T>(v);
    v = act_value(P.act, v);
    if (P.res) v += to_f32(static_cast<const T *>(P.res)[m * P.ldr + n]);
    static_cast<T *>(P.y)[m * P.ldy + n] = from_f32<T>(v);
}

// One 128 x bn tile of D per cluster; the `splits` CTAs of the cluster share
// its reduction (contiguous runs of 64-step blocks).  Each CTA leaves its fp32
// partial tile in its own shared memory; after a cluster barrier CTA c reads
// the c-th part of the tile from all of them through distributed shared
// memory, always in rank order, and stores it.  So a product with few tiles
// uses all SMs in one launch, without a workspace, and gives the same bits
// each time.
template <typename T>
__global__ void __launch_bounds__(kLinThreads) linear_tile_kernel(const __grid_constant__ LinParams P) {
    extern __shared__ uint8_t lin_smem_raw[];
    __shared__ uint64_t full[kLinMaxStages], empty[kLinMaxStages], done;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    uint8_t *smem = lin_smem_raw + ((1024u - (smem_u32(lin_smem_raw) & 1023u)) & 1023u);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = blockIdx.x % P.splits, tile = blockIdx.x / P.splits;
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

    // partial tile -> shared memory as [outer][inner], the output's row index
    // (token) outer: i outer in the plain form, j outer in the swapped one
    float *part = reinterpret_cast<float *>(smem);
    const int ld = P.swap ? kLinRows : P.bn + 1;   // odd stride: lanes write distinct banks
    if (warp >= 2) {
        mbar_wait(&done, 0, kLinTimeoutNs, abort);
        tc_fence_after();
        const int quad = warp & 3, i = quad * 32 + lane;
        for (int c = 0; c < P.bn; c += 16) {
            uint32_t r[16];
            tc_ld_32x32b_x16(tmem + (static_cast<uint32_t>(quad * 32) << 16) + c, r);
            tc_wait_ld();
            if (P.swap) {
#pragma unroll
                for (int q = 0; q < 16; ++q) part[(c + q) * ld + i] = __uint_as_float(r[q]);
            } else {
#pragma unroll
                for (int q = 0; q < 16; ++q) part[i * ld + c + q] = __uint_as_float(r[q]);
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, tmem_cols);
    }
    if (P.splits > 1) cluster_sync();

    const int outer = P.swap ? P.bn : kLinRows, inner = P.swap ? kLinRows : P.bn;
    const int m0 = P.swap ? j0 : i0, n0 = P.swap ? i0 : j0;
    const int M = P.swap ? P.J : P.I, N = P.swap ? P.I : P.J;
    const int o0 = outer * rank / P.splits, o1 = min(outer * (rank + 1) / P.splits, M - m0);
    const int width = min(inner, N - n0);
    for (int o = o0 + warp; o < o1; o += kLinThreads / 32)
        for (int n = lane; n < width; n += 32) {
            float v;
            if (P.splits == 1) {
                v = part[o * ld + n];
            } else {
                const uint32_t at = smem_u32(part + o * ld + n);
                v = 0.f;
                for (int c = 0; c < P.splits; ++c) v += ld_cluster_f32(map_to_rank(at, c));
            }
            lin_store<T>(P, v, static_cast<int64_t>(m0) + o, n0 + n);
        }
    if (P.splits > 1) cluster_sync();   // no CTA leaves while others read its part
}

// Copy of a matrix whose rows are not multiples of 16 bytes into rows of
// round_up(cols, 8) elements (the tensor maps' stride rule).
static __global__ void linear_pack_kernel(const uint16_t *src, int64_t ld, int64_t rows, int32_t cols, uint16_t *dst,
                                          int64_t ldd) {
    const int64_t per = ldd / 8, n = rows * per;
    for (int64_t e = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; e < n;
         e += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t r = e / per;
        const int c0 = static_cast<int>(e % per) * 8;
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (c0 + q < cols) w[q / 2] |= static_cast<uint32_t>(src[r * ld + c0 + q]) << (16 * (q & 1));
        *reinterpret_cast<uint4 *>(dst + r * ldd + c0) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// dz = g * act'(z) (rounded to the operand type of the products) and the
// column sums of the unrounded dz over a slab of rows.  A block is 32 lanes x
// 8 row groups; a lane owns 8 columns.  VEC: whole 16-byte loads.
constexpr int kDzRows = 8;
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) linear_dz_kernel(const T *g, int64_t ldg, const T *z, int64_t ldz, int32_t M,
                                                        int32_t N, int32_t act, T *dz, int64_t lddz, float *part,
                                                        int32_t slab) {
    __shared__ float sums[kDzRows][32][9];
    const int lane = threadIdx.x % 32, ty = threadIdx.x / 32;
    const int c0 = (blockIdx.x * 32 + lane) * 8;
    const int r1 = static_cast<int>(min(static_cast<int64_t>(M), (blockIdx.y + static_cast<int64_t>(1)) * slab));
    float acc[8] = {};
    if (c0 < N) {
        for (int64_t r = static_cast<int64_t>(blockIdx.y) * slab + ty; r < r1; r += kDzRows) {
            float v[8];
            if (VEC && c0 + 8 <= N) {
                Vec<T>::widen(*reinterpret_cast<const uint4 *>(g + r * ldg + c0), v);
                if (z) {
                    float zv[8];
                    Vec<T>::widen(*reinterpret_cast<const uint4 *>(z + r * ldz + c0), zv);
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[q] *= act_slope(act, zv[q]);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    v[q] = 0.f;
                    if (c0 + q < N) {
                        v[q] = to_f32(g[r * ldg + c0 + q]);
                        if (z) v[q] *= act_slope(act, to_f32(z[r * ldz + c0 + q]));
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] += v[q];
            if (dz) *reinterpret_cast<uint4 *>(dz + r * lddz + c0) = Vec<T>::narrow(v);   // lddz = round_up(N, 8)
        }
    }
    if (part == nullptr) return;
#pragma unroll
    for (int q = 0; q < 8; ++q) sums[ty][lane][q] = acc[q];
    __syncthreads();
    // 256 columns of the block, one per thread
    const int l = threadIdx.x / 8, q = threadIdx.x % 8, c = (blockIdx.x * 32 + l) * 8 + q;
    if (c < N) {
        float s = 0.f;
        for (int k = 0; k < kDzRows; ++k) s += sums[k][l][q];
        part[static_cast<int64_t>(blockIdx.y) * N + c] = s;
    }
}

// gb[n] = sum of the slabs' partial sums, in slab order.
static __global__ void linear_bias_grad_kernel(const float *part, int32_t slabs, int32_t N, float *gb) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= N) return;
    float s[4] = {};
    int k = 0;
    for (; k + 4 <= slabs; k += 4)
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] += part[static_cast<int64_t>(k + q) * N + c];
    for (; k < slabs; ++k) s[0] += part[static_cast<int64_t>(k) * N + c];
    gb[c] = (s[0] + s[1]) + (s[2] + s[3]);
}

}  // namespace mqc
