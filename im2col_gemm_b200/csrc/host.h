// host.h -- host helpers shared by the library's translation units: error
// reporting, device properties, and the encoder of TMA tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/mqc.h"
#include "common.cuh"

namespace mqc {

// Records the one-line reason of the calling thread's last failure and
// returns `s`.
mqc_status fail(mqc_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
mqc_status cuda_fail(cudaError_t e, const char *what);

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The current device: its ordinal, SM count and shared memory per block.
// Fails on anything but sm_100.
struct DeviceLimits {
    int device, sms, max_smem;
};
mqc_status device_limits(DeviceLimits *out);

// Tensor map of a row-major matrix of 2-byte elements, `rows` x `cols` with
// row stride `ld` elements: boxes of `box_bytes` (128 or 64, with the swizzle
// of that width) x `box_rows` rows; coordinates are (byte, row).  Bytes beyond the
// matrix read as zero.  `base` and ld * 2 must be multiples of 16.
mqc_status encode_matrix_map(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int64_t ld,
                             int box_rows, int box_bytes = 128);

// Reads and clears the device error word of the linear kernels (each
// translation unit has its own word).
cudaError_t linear_take_device_error(int *value);

inline FastDiv make_fastdiv(int32_t d) {
    FastDiv f;
    f.d = static_cast<uint32_t>(std::max(1, d));
    f.l = 0;
    while ((1ull << f.l) < f.d) ++f.l;
    f.m = static_cast<uint32_t>(((1ull << 32) * ((1ull << f.l) - f.d)) / f.d + 1);
    return f;
}

// The configuration of a launch in clusters; `after`: behind the call's previous
// kernel, which it waits for by itself (wait_previous).
struct Launch {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[2];
    Launch(int64_t grid, int threads, int cluster, size_t smem, bool after, cudaStream_t stream) {
        cfg.gridDim = dim3(static_cast<unsigned>(grid));
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cfg.attrs = at;
        if (cluster > 0) {
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = cluster;
            at[0].val.clusterDim.y = 1;
            at[0].val.clusterDim.z = 1;
            cfg.numAttrs = 1;
        }
        if (after) {
            at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            at[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
        }
    }
    Launch(const Launch &) = delete;
};

inline bool act_ok(int act) { return act >= MQC_ACT_NONE && act <= MQC_ACT_GELU; }
inline int dtype_bytes(int dtype) { return dtype == MQC_F32 ? 4 : 2; }

}  // namespace mqc
