// serving_checks.cuh -- host-side argument checks that the entries of the serving operators share.
#pragma once

#include "../common.cuh"

namespace tsv {
tsv_status report_error(tsv_status s, const char* fmt, ...);
}  // namespace tsv

namespace {
using tsv::report_error;

inline int device_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return 148;
    return sms;
}

inline bool pow2_in(int x, int lo, int hi) { return x >= lo && x <= hi && (x & (x - 1)) == 0; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline int log2i(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
}

inline tsv_status launch_status(cudaError_t e, const char* what) {
    return e == cudaSuccess ? TSV_OK : report_error(TSV_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

inline tsv_status check_cache_shape(int Hkv, int D, int block_size, int num_blocks, tsv_dtype dtype) {
    if (Hkv < 1 || num_blocks < 1) return report_error(TSV_ERR_ARG, "bad sizes Hkv=%d num_blocks=%d", Hkv, num_blocks);
    if (D != 64 && D != 128) return report_error(TSV_ERR_UNSUPPORTED, "head dim %d not in {64, 128}", D);
    if (!pow2_in(block_size, 8, 128)) return report_error(TSV_ERR_UNSUPPORTED, "block_size %d not a power of two in [8,128]", block_size);
    if (dtype != TSV_BF16 && dtype != TSV_F32) return report_error(TSV_ERR_ARG, "bad dtype %d", (int)dtype);
    return TSV_OK;
}

// The kernels hold the offsets within a token's row in 32 bits (and three rows of the caches on).
inline tsv_status check_row(int heads, int D) {
    if ((long long)heads * D > (1LL << 28)) return report_error(TSV_ERR_UNSUPPORTED, "a row of %d heads of %d exceeds 2^28 elements", heads, D);
    return TSV_OK;
}
}  // namespace
