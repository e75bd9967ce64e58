// adapters.cuh -- what the low-rank adapter kernels share: the layout of a plan (the tokens of a
// batch ordered by adapter), the operands of a call and the launchers of the kernel files.
#pragma once

#include "qlin_common.cuh"

namespace qlin {

// Tokens of one adapter are cut into tiles of 8 (decode) and of 128 (tensor-core kernels).
constexpr int kTileS = 8;
constexpr int kTileL = 128;
constexpr int64_t kMaxAdapters = 1024;      // the plan kernel's counters fill 32 x (L + 1) ints of shared memory
constexpr int64_t kMaxPlanTokens = 1 << 20;
constexpr int kMaxRank = 128;

// One tile: tokens perm[start .. start + count - 1] of `adapter` (the number of adapters for the
// tokens without one).  first: the tile's first token when its tokens are consecutive, else -1.
struct __align__(16) AdapterTile {
    int adapter, start, count, first;
};

// A plan is a device buffer of int32: a header, where each adapter's tokens start in perm and its
// tiles start in the two lists, perm, and the lists.  Tokens without an adapter come last.
struct PlanView {
    int* head;            // [8]: M, L, tiles of 8, tiles of 128, then both without the last segment's
    int* seg;             // [L + 2] first position of adapter i; [L] the tokens without one; [L + 1] = M
    int* tile_l0;         // [L + 2] first 128-tile of adapter i
    int* perm;            // [M] tokens by adapter, ascending inside one
    AdapterTile* tiles_s; // [max_tiles(M, L, 8)]
    AdapterTile* tiles_l; // [max_tiles(M, L, 128)]
};

__host__ __device__ inline int64_t plan_up4(int64_t v) { return (v + 3) & ~int64_t(3); }
// at most one partly filled tile for each segment that holds a token
__host__ __device__ inline int64_t max_tiles(int64_t M, int64_t L, int64_t t) { return M / t + (M < L + 1 ? M : L + 1); }
__host__ __device__ inline int64_t plan_ints(int64_t M, int64_t L)
{
    return 8 + 2 * plan_up4(L + 2) + plan_up4(M) + 4 * (max_tiles(M, L, kTileS) + max_tiles(M, L, kTileL));
}
__host__ __device__ inline PlanView plan_view(const void* plan, int64_t M, int64_t L)
{
    PlanView v;
    int* p = static_cast<int*>(const_cast<void*>(plan));
    v.head = p;
    v.seg = p + 8;
    v.tile_l0 = v.seg + plan_up4(L + 2);
    v.perm = v.tile_l0 + plan_up4(L + 2);
    v.tiles_s = reinterpret_cast<AdapterTile*>(v.perm + plan_up4(M));
    v.tiles_l = v.tiles_s + max_tiles(M, L, kTileS);
    return v;
}

struct AdapterFwdArgs {
    const void* x;        // [M][K]
    const void* a;        // [L][R][K]
    const void* b;        // [L][N][R]
    const float* scales;  // [L]
    const void* base;     // [M][N] or null (zeros); may be out
    void* out;            // [M][N]
    float* u;             // [M][R] or null
    qlin_dtype dt;
    int64_t M, K, N, L, R;
    PlanView plan;
    void* ws;
};

struct AdapterBwdArgs {
    const void* dy;        // [M][N]
    const void* a;
    const void* b;
    const float* scales;
    const float* u;        // [M][R]
    const void* x;         // [M][K] of dt, or null:
    const int8_t* q;       // [M][K] int8 and
    const float* q_scale;  // [K / g][M]
    int g;
    const void* dx_base;   // [M][K] or null; may be dx
    void* dx;              // [M][K] or null (not wanted)
    void* da;              // [L][R][K]
    void* db;              // [L][N][R]
    qlin_dtype dt;
    int64_t M, K, N, L, R;
    PlanView plan;
    void* ws;
};

cudaError_t launch_adapters_plan(const int32_t* ids, int64_t M, int64_t L, void* plan, cudaStream_t st);

// Any type, size and alignment (k_adapters.cu).
size_t adapters_simt_workspace(int64_t M, int64_t N, int64_t K, int64_t R);
cudaError_t launch_adapters_forward_simt(const AdapterFwdArgs& a, cudaStream_t st);
cudaError_t launch_adapters_backward_simt(const AdapterBwdArgs& a, cudaStream_t st);


// Tensor-core kernels (k_adapters_tc.cu): bf16 and fp16, K and N multiples of 8, R of 4, every tensor
// 16-byte aligned.
bool adapters_tc_takes(const AdapterFwdArgs& a);
bool adapters_tc_takes(const AdapterBwdArgs& a);
size_t adapters_tc_workspace(int64_t M, int64_t N, int64_t L, int64_t R);
cudaError_t launch_adapters_forward_tc(const AdapterFwdArgs& a, cudaStream_t st, const DeviceInfo& dev);
cudaError_t launch_adapters_backward_tc(const AdapterBwdArgs& a, cudaStream_t st, const DeviceInfo& dev);

// Host: a 3-D tensor map over dense [dim2][dim1][dim0] elements of elem_bytes, box {box0, box1, 1},
// 128-byte swizzle, zero fill (qlin_abi.cu).
bool encode_tmap_3d(CUtensorMap* tm, CUtensorMapDataType dt, const void* base, uint64_t dim0, uint64_t dim1,
                    uint64_t dim2, uint64_t elem_bytes, uint32_t box0, uint32_t box1);

// Loads the box at (c0, c1, c2) of a 3-D tensor map into this CTA's shared memory.
QLIN_DEV void tma_load_3d(void* smem_dst, const CUtensorMap* tmap, int c0, int c1, int c2, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}

}  // namespace qlin
