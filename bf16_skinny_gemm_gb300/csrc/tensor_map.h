// The encoder of tensor maps, and maps of BF16 arrays for the operators of sgemm_layers.h.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace sk {

inline PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *q = nullptr;
        cudaDriverEntryPointQueryResult res;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault, &res) != cudaSuccess ||
            res != cudaDriverEntryPointSuccess)
            q = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(q);
    }();
    return fn;
}

// [n2][n1][n0] elements with strides s2, s1 and 1 (elements), copied in boxes of b1 rows x `deep` chunks of 64
// elements, each chunk's rows by themselves and 128-byte swizzled; what lies outside reads as 0.  With `even` (n0 a
// multiple of 64) the map is [n2][n0 / 64][n1][64], else [n2][1][n1][n0] with one chunk a box.  A stride along a
// dimension of one is of no account (a map's strides have to be multiples of 16 bytes below 2^40).
inline bool map_4d(CUtensorMap *map, const void *base, long long n0, long long n1, long long n2, long long s1, long long s2,
                   int b1, int deep, bool even, CUtensorMapL2promotion promote) {
    auto enc = map_encoder();
    if (!enc) return false;
    if (n1 == 1) s1 = (n0 + 7) / 8 * 8;
    if (n2 == 1) s2 = s1;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(even ? 64 : n0), static_cast<cuuint64_t>(n1),
                                static_cast<cuuint64_t>(even ? n0 / 64 : 1), static_cast<cuuint64_t>(n2)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(s1) * 2, 128, static_cast<cuuint64_t>(s2) * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(even ? deep : 1), 1}, ones[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promote, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

constexpr long long kMapStride = 1LL << 38;  // elements: strides a map can hold, with room to spare

}  // namespace sk
