// What the persistent products on 128-byte swizzled tiles share: operand
// descriptors, the way of a tile's output to memory, and tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "tc_common.cuh"
#include "tc_ptx.cuh"

using namespace tc;

namespace {

#define TILE_FAIL(code, ...)       \
    do {                           \
        sg_set_error(__VA_ARGS__); \
        return code;               \
    } while (0)

constexpr uint32_t kBox = 8192;          // one TMA box: 64 rows of 128 bytes
constexpr uint32_t kStgWarp = 4096;      // an epilogue warp's outputs on their way: two boxes of 32 x 32

// Descriptors of an operand's tile at shared address `base`: the low word, to
// which stages (bytes / 16) and K steps are added, the high word, and the step.
// K-major: rows of 128 bytes of K, 8 rows to a swizzle atom.  MN-major: boxes
// of 64 rows (128 bytes) by 64 K, kBox apart.  Worked out once for a tile: the
// thread that issues the MMAs has little time for each.
struct OpDesc {
    uint32_t lo, hi, step;

    __device__ __forceinline__ OpDesc(uint32_t base, bool mn)
    {
        const uint64_t d = sdesc(base, mn ? kBox : 16, 1024, kLayoutSW128);
        lo = (uint32_t)d;
        hi = (uint32_t)(d >> 32);
        step = mn ? 2048 / 16 : 32 / 16;
    }
    __device__ __forceinline__ uint64_t at(uint32_t stage, int ks) const
    {
        return (uint64_t)hi << 32 | (lo + stage + ks * step);
    }
};

__device__ __forceinline__ uint32_t pack16(float a, float b, bool f16)
{
    return f16 ? pack2_f16(a, b) : pack2(a, b);
}

// 32 columns (16 packed words) of this warp's 32 rows to global memory by TMA,
// from one of its two boxes while the other is filled: rows of 64 bytes, their
// 16-byte units swizzled.  Lane 0 issues the store, if `in`.
__device__ __forceinline__ void store_box(const CUtensorMap *map, int x, int y, bool in, uint8_t *box, int lane,
                                          const uint32_t (&w)[16])
{
    if (lane == 0)
        bulk_wait_read<1>();
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4 *>(box + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
        if (in)
            tma_store_2d(map, x, y, smem_u32(box));
        bulk_commit();
    }
}

// ---------------------------------------------------------------- host
std::atomic<PFN_cuTensorMapEncodeTiled_v12000> g_encode_tile{nullptr};

// row-major matrix in boxes of box_rows x 128 bytes, 128-byte swizzle;
// `narrow`: 64 bytes, 64-byte swizzle
sg_status map_of(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, int64_t ld, int elem,
                 const char *what, uint32_t box_rows = 64, bool narrow = false)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = g_encode_tile.load(std::memory_order_acquire);
    if (!enc) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !fn) {
            cudaGetLastError();
            TILE_FAIL(SG_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
        }
        enc = (PFN_cuTensorMapEncodeTiled_v12000)fn;
        g_encode_tile.store(enc, std::memory_order_release);
    }
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(ld * elem)};
    cuuint32_t box[2] = {(narrow ? 64u : 128u) / (uint32_t)elem, box_rows};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(m, elem == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                               : elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16
                                           : CU_TENSOR_MAP_DATA_TYPE_UINT32, 2,
                           const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           narrow ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        TILE_FAIL(SG_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", what, (int)r);
    return SG_OK;
}

bool tma_ok(const void *p, int64_t ld, int64_t es) { return ((uintptr_t)p & 15) == 0 && (ld * es) % 16 == 0; }

}  // namespace
