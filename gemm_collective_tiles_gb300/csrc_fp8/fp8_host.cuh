// Host side that products share: errors, launches, argument checks, operand
// layouts, tensor maps.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "gemm_collective_tiles.h"
#include "fp8_repack.cuh"

namespace {

using namespace gct;
using namespace gct::fp8;

constexpr size_t WS_HEADER = 256;
constexpr unsigned long long DEFAULT_WAIT_NS = 2000000000ull;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

std::mutex g_mu;
EncodeTiledFn g_encode = nullptr;

int cuda_fail(const char* what, int code) {
    static const bool on = [] {
        const char* e = std::getenv("IRIS_B200_DEBUG");
        return e && e[0] && e[0] != '0';
    }();
    if (on) std::fprintf(stderr, "[iris_b200] %s failed: %d\n", what, code);
    return IRIS_ECUDA;
}

// the driver's tensor-map encoder; g_mu is held
int find_encode() {
    if (g_encode) return IRIS_OK;
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn)
        return cuda_fail("cuTensorMapEncodeTiled entry point", -1);
    g_encode = reinterpret_cast<EncodeTiledFn>(fn);
    return IRIS_OK;
}

// Every kernel here may start while the one before it in the stream still runs
// (it waits for that one's end before it touches memory), which hides its launch
// and set-up behind its forerunner's last CTAs: one token's quantisation 1.5 ->
// 1.3 us, 333 x 1000 x 1111 9.9 -> 9.2, 8192^3 388 -> 380.
cudaLaunchConfig_t launch_config(unsigned grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                                 cudaLaunchAttribute (&attr)[2]) {
    cudaLaunchConfig_t lc;
    std::memset(&lc, 0, sizeof(lc));
    lc.gridDim = dim3(grid);
    lc.blockDim = dim3(threads);
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    std::memset(attr, 0, sizeof(attr));
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        lc.numAttrs = 2;
    }
    return lc;
}
template <typename... Params, typename... Args>
int launch(const char* what, void (*kernel)(Params...), const cudaLaunchConfig_t& lc, Args... args) {
    const cudaError_t e = cudaLaunchKernelEx(&lc, kernel, static_cast<Params>(args)...);
    return e == cudaSuccess ? IRIS_OK : cuda_fail(what, static_cast<int>(e));
}

template <typename Kernel>
int setup_kernel(Kernel kernel, int* clusters, int lg_lo, int lg_hi, int threads, size_t smem, int regs, int sms) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return cuda_fail("cudaFuncSetAttribute (products)", static_cast<int>(e));
    // the warpgroups' register shares must fit in what the launch allots, or
    // a warpgroup would wait for registers that never come
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return cuda_fail("cudaFuncGetAttributes", static_cast<int>(e));
    if (fa.numRegs * threads < regs) return cuda_fail("register shares of the products", fa.numRegs);
    for (int lg = lg_lo; lg <= lg_hi; ++lg) {
        clusters[lg] = sms;
        if (lg == 0) continue;
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t lc = launch_config(sms >> lg << lg, threads, smem, 1 << lg, nullptr, attr);
        e = cudaOccupancyMaxActiveClusters(&clusters[lg], kernel, &lc);
        if (e != cudaSuccess || clusters[lg] < 1) return cuda_fail("cudaOccupancyMaxActiveClusters", static_cast<int>(e));
    }
    return IRIS_OK;
}
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
int dtype_size(int t) { return t == IRIS_F32 ? 4 : 2; }

bool dims_ok(int64_t M, int64_t N, int64_t K) {
    // 128-rounded sizes stay below 2^31
    const int64_t lim = (int64_t(1) << 31) - 512;
    return M >= 0 && N >= 0 && K >= 0 && M <= lim && N <= lim && K <= lim;
}
bool dtype16(int t) { return t == IRIS_F16 || t == IRIS_BF16; }
bool dtype_ok(int t) { return dtype16(t) || t == IRIS_F32; }
bool fp8_ok(int t) { return t == IRIS_E4M3 || t == IRIS_E5M2; }

// a matrix that is read: pointer (unless empty), no negative stride, element alignment
int check_in(const iris_b200_mat* m, int64_t rows, int64_t cols, int elem) {
    if (!m || m->row_stride < 0 || m->col_stride < 0) return IRIS_EINVAL;
    if (rows == 0 || cols == 0) return IRIS_OK;
    if (!m->data) return IRIS_EINVAL;
    return reinterpret_cast<uintptr_t>(m->data) % elem ? IRIS_EALIGN : IRIS_OK;
}
// a matrix that is written: also no two elements at one address
int check_out(const iris_b200_mat* m, int64_t rows, int64_t cols, int elem) {
    const int rc = check_in(m, rows, cols, elem);
    if (rc) return rc;
    const int64_t r = m->row_stride, c = m->col_stride;
    if (rows > 1 && r < 1) return IRIS_EINVAL;
    if (cols > 1 && c < 1) return IRIS_EINVAL;
    if (rows > 1 && cols > 1 && r <= c * (cols - 1) && c <= r * (rows - 1)) return IRIS_EINVAL;
    return IRIS_OK;
}

// How the tensor memory accelerator can read a matrix in place: rows of unit
// stride on a 16-byte base and pitch.
bool tma_rows(const void* data, int64_t row_stride, int64_t col_stride, int64_t rows, int64_t cols, int elem) {
    return aligned16(data) && (col_stride == 1 || cols == 1) &&
           (rows == 1 || (row_stride >= cols && row_stride * elem % 16 == 0 && row_stride * elem < (int64_t(1) << 40)));
}
int64_t packed_pitch(int64_t cols, int elem) { return static_cast<int64_t>(round_up(cols * elem, 16)) / elem; }

// Operand as it will be read: in place, or copied into rows of whole 16 bytes.
struct Operand {
    const void* data;
    int64_t rows, cols, pitch;  // rows of unit-stride elements
    bool transposed;            // its rows are the matrix's columns
    bool copy;
    size_t copy_bytes;
};
Operand resolve_operand(const iris_b200_mat* m, int64_t rows, int64_t cols, int elem, bool may_transpose) {
    Operand o{m->data, rows, cols, m->row_stride, false, false, 0};
    if (tma_rows(m->data, m->row_stride, m->col_stride, rows, cols, elem)) {
        if (rows == 1) o.pitch = packed_pitch(cols, elem);
        return o;
    }
    if (may_transpose && tma_rows(m->data, m->col_stride, m->row_stride, cols, rows, elem)) {
        o = Operand{m->data, cols, rows, m->col_stride, true, false, 0};
        if (cols == 1) o.pitch = packed_pitch(rows, elem);
        return o;
    }
    // columns of unit stride are copied as the rows that they are
    if (may_transpose && rows > 1 && m->row_stride == 1 && m->col_stride != 1) o = Operand{m->data, cols, rows, 0, true, false, 0};
    o.copy = true;
    o.pitch = packed_pitch(o.cols, elem);
    o.copy_bytes = round_up(static_cast<size_t>(o.rows) * o.pitch * elem, 256);
    return o;
}
template <typename E>
int launch_repack(const iris_b200_mat* m, Operand& o, void* dst, int sms, cudaStream_t stream) {
    const int64_t rs = o.transposed ? m->col_stride : m->row_stride, cs = o.transposed ? m->row_stride : m->col_stride;
    constexpr int64_t elem = sizeof(E);
    const bool by_rows = cs == 1 || o.cols == 1;
    const int64_t tiles = by_rows ? cdiv(o.rows, COPY_ROWS) * cdiv(o.pitch * elem, 512) : cdiv(o.rows, 32) * cdiv(o.cols, 32);
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t lc = launch_config(static_cast<unsigned>(std::min<int64_t>(tiles, int64_t(sms) * 8)), 256, 0, 1, stream, attr);
    const int rc = by_rows ? launch("repack launch", repack_rows_kernel, lc, static_cast<const uint8_t*>(m->data), rs * elem,
                                    static_cast<uint8_t*>(dst), o.pitch * elem, o.rows, o.cols * elem)
                           : launch("repack launch", repack_kernel<E>, lc, static_cast<const E*>(m->data), rs, cs,
                                    static_cast<E*>(dst), o.pitch, o.rows, o.cols);
    if (rc) return rc;
    o.data = dst;
    return IRIS_OK;
}

// A tensor map.  The driver's call wants the calling thread to have a context,
// which runtime calls give it; a thread that has made none that does (autograd's,
// whose first work may be a product) is given the current device's here.
CUresult encode(CUtensorMap* m, CUtensorMapDataType dt, cuuint32_t rank, const void* data, const cuuint64_t* dims,
                const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapL2promotion l2) {
    const cuuint32_t es[3] = {1, 1, 1};
    auto call = [&] {
        return g_encode(m, dt, rank, const_cast<void*>(data), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, l2, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    const CUresult r = call();
    int dev = 0;
    if (r != CUDA_ERROR_INVALID_CONTEXT || cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return r;
    return call();
}
int make_map_2d(CUtensorMap* m, CUtensorMapDataType dt, int elem, const Operand& o, uint32_t b0, uint32_t b1) {
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(o.cols), static_cast<cuuint64_t>(o.rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(o.pitch) * elem};
    cuuint32_t box[2] = {b0, b1};
    const CUresult r = encode(m, dt, 2, o.data, dims, strides, box, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    return r == CUDA_SUCCESS ? IRIS_OK : cuda_fail("cuTensorMapEncodeTiled (operand)", static_cast<int>(r));
}
// 16-bit rows as groups of 64 columns, {64, row, column / 64}: a box of 64 rows
// of `groups` groups, 8192 bytes each
int make_map_groups(CUtensorMap* m, CUtensorMapDataType dt, const Operand& o, uint32_t groups) {
    cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(o.rows), static_cast<cuuint64_t>(o.cols / 64)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(o.pitch) * 2, 128};
    cuuint32_t box[3] = {64, 64, groups};
    const CUresult r = encode(m, dt, 3, o.data, dims, strides, box, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    return r == CUDA_SUCCESS ? IRIS_OK : cuda_fail("cuTensorMapEncodeTiled (groups of columns)", static_cast<int>(r));
}
// out {n, row} with a box of 128 bytes x 32 rows
int make_store_map(CUtensorMap* m, int t, const void* data, int64_t N, int64_t M, int64_t pitch) {
    const int elem = dtype_size(t);
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * elem};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / elem), 32};
    const CUtensorMapDataType dt = t == IRIS_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : t == IRIS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                   : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUresult r = encode(m, dt, 2, data, dims, strides, box, CU_TENSOR_MAP_L2_PROMOTION_NONE);
    return r == CUDA_SUCCESS ? IRIS_OK : cuda_fail("cuTensorMapEncodeTiled (output)", static_cast<int>(r));
}

}  // namespace
