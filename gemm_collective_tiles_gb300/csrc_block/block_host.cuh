// What the host sides of the ops around linear layers share.
#pragma once
#include "../csrc_fp8/fp8_host.cuh"
#include "block_elem.cuh"

namespace {

using namespace gct::block;

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// an optional vector
int check_vec(const void* data, int type) {
    if (!data) return IRIS_OK;
    if (!dtype_ok(type)) return IRIS_EINVAL;
    return aligned(data, dtype_size(type)) ? IRIS_OK : IRIS_EALIGN;
}
Mat mat_of(const iris_b200_mat& m) { return Mat{m.data, m.row_stride, m.col_stride}; }
// rows of unit stride on 16 bytes
bool rows16(const iris_b200_mat& m, int64_t rows, int64_t cols, int elem) {
    return !m.data || (aligned16(m.data) && (m.col_stride == 1 || cols == 1) && (rows <= 1 || m.row_stride * elem % 16 == 0));
}
int sm_count(int* sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return IRIS_ECUDA;
    return IRIS_OK;
}

}  // namespace
