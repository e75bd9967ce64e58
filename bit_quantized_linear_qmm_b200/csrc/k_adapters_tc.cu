// k_adapters_tc.cu -- low-rank adapters on the tensor cores, bf16 and fp16 (sm_100a).
//
//   narrow   h[m] = A_i x[m]  (forward)  or  v[m] = s_i B_i^T dy[m]  (backward)
//   wide     out[m] = base[m] + s_i B_i h[m]   or   dx[m] = dx_base[m] + A_i^T v[m]
//   grams    dB_i = s_i sum_m dy[m] u[m]^T,  dA_i^T = sum_m x[m] v[m]^T
//   decode   both products of the forward pass for few tokens, in one launch
//
// The first three are tcgen05 kernels.  Each moves one long activation row in (or one in and one
// out) for every token and does 2 to 4 R products a value, R <= 128, so memory bounds them; the
// tensor cores and the threads only have to keep up.  Tokens are taken in tiles of 128 of one
// adapter (the plan's list).  A tile whose tokens are consecutive is read in tensor-map boxes of 64
// rows, any other by tile::gather4, four rows an instruction: no thread touches the data before
// the tensor cores.  A thread issues a box in about 150 cycles and a warp a gather in about 86 (its
// lanes take turns), so four warps share a stage's copies (one thread took 940 cycles for the six of
// a gram step, longer than anything else in it).
//
// h, u and v enter their second product as two 16-bit halves, hi = round(h) and lo = round(h - hi):
// 2^-16 of the value at most (fp16: or 2^-39 of the largest under one scale, half of fp16's smallest
// step, where that is more), and two MMAs instead of one.  They are kept in slots, [tile][128][Rq]
// (Rq = R rounded up to 16), zero where there is no token or rank, hi and lo apart.  fp16 halves
// are scaled by a power of two that puts the largest value of the row (wide) or of the adapter
// (grams) in [2^14, 2^15), undone on the fp32 sum; bf16 has fp32's range and needs none.
//
// Every mbarrier wait is bounded: on expiry the kernel records the timeout, every role stops, MMAs
// and copies in flight are waited for and TMEM is freed.
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "adapters.cuh"

namespace qlin {
namespace {

constexpr uint32_t kAtom = 64 * 128;  // a 64-row x 128-byte swizzled block
constexpr int kMaxSplit = 16;         // CTAs of a cluster (beyond 8: allowed on this GPU, not portable)

// ------------------------------------------------------------------------------------ helpers

QLIN_DEV void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// this shared-memory address in CTA `rank` of the cluster
QLIN_DEV uint32_t peer_smem(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
QLIN_DEV float4 ld_peer_v4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}
QLIN_DEV float ld_peer(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}
QLIN_DEV void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
QLIN_DEV bool aborted(int* flag) { return *reinterpret_cast<volatile int*>(flag) != 0; }

template <typename T> struct Is16 { static constexpr int f16 = 0; };
template <> struct Is16<__half> { static constexpr int f16 = 1; };

// (a, b) as hi + lo pairs.  A half that is infinite has no remainder.
template <typename T>
QLIN_DEV void split2(float a, float b, uint32_t& hi, uint32_t& lo)
{
    constexpr int f16 = Is16<T>::f16;
    hi = pack_h16x2(a, b, f16);
    const float ra = a - h16_to_float(hi, f16), rb = b - h16_to_float(hi >> 16, f16);
    lo = pack_h16x2(fabsf(ra) <= 3.4e38f ? ra : 0.f, fabsf(rb) <= 3.4e38f ? rb : 0.f, f16);
}

// Power of two that puts a finite m in [2^14, 2^15) (1 for 0), for fp16 halves; 1 for bf16.  The
// exponent is clamped so that the factor and its inverse are normal.
template <typename T>
QLIN_DEV void half_scale(float m, float& to, float& back)
{
    to = back = 1.f;
    if constexpr (Is16<T>::f16) {
        if (m > 0.f) {
            int e = (int)(__float_as_uint(m) >> 23) - 127 - 14;  // m 2^-e in [2^14, 2^15)
            e = e < -120 ? -120 : e > 120 ? 120 : e;
            to = __uint_as_float((uint32_t)(127 - e) << 23);
            back = __uint_as_float((uint32_t)(127 + e) << 23);
        }
    }
}
QLIN_DEV float finite_abs(float v)
{
    const float a = fabsf(v);
    return a <= 3.4028235e38f ? a : 0.f;
}

// Sorted-token views that the kernels share.
struct Common {
    PlanView plan;
    int64_t M, slots;       // slots: 128 for each tile of the plan's bound
    int L, R, Rq;
    int Rb;                 // ranks of a row of B as the tensor maps read it
    void* b_pad;            // where R % 8 is 4: B with rows of Rb = R + 4 ranks
    uint16_t* row_halves;   // [2][slots][Rq]: hi and lo of h (forward) or v, for the wide product
    uint16_t* v_halves;     // [2][slots][Rq]: of v for the grams (bf16: the same)
    uint16_t* u_halves;     // [2][slots][Rq]: of u for the grams
    float* row_back;        // [slots], fp16: what undoes a row's scale
    float* v;               // [slots][Rq], fp16 backward: v itself
    float* tile_max;        // [tiles][kMaxSplit][2], fp16 backward: largest finite |v| and |u| of a CTA's rows
    unsigned* status;
};

// Four rows of a 2-D tensor map (box {64, 1}) into consecutive 128-byte rows.
QLIN_DEV void tma_gather4(uint32_t dst, const CUtensorMap* tm, int c0, const int4& r, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(smem_u32(bar))
        : "memory");
}

// A matrix of token rows: boxes of 64 rows, and single rows for gathers.
struct RowMaps {
    CUtensorMap box, row;
};

// One thread: a box of 64 rows from row `first`, 128 bytes of each from column c0.
QLIN_DEV void load_box(uint32_t dst, const CUtensorMap* m, int c0, int first, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(first), "r"(smem_u32(bar))
        : "memory");
}

// Tokens of rows 4 i .. 4 i + 3 of positions [start, start + count); past the end the first one (its
// row is read and never used, or zeroed).
QLIN_DEV int4 row_tokens(const PlanView& v, int start, int count, int i)
{
    int t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        t[e] = v.perm[start + (4 * i + e < count ? 4 * i + e : 0)];
    return make_int4(t[0], t[1], t[2], t[3]);
}

// ------------------------------------------------------------------------------------ narrow

// One cluster for each tile of 128 tokens: its CTAs split the contraction, each accumulating
// [128][Rq] in tensor memory over its steps of 64; the partial sums meet through distributed shared
// memory, CTA j adding the parts of rows 128 j / z .. in order, so h is written once and the order
// of every sum is fixed.
//   warps 0..3   the loads: activation rows, and (warp 0) the factor -- forward A_i [Rq rows][64 k],
//                K-major; backward B_i [64 n][R], MN-major -- from a 3-D map, so that rows and
//                columns past the adapter's own are zeros
//   warp 4       tensor memory, the MMAs (M = 128, N = Rq, K = 16)
//   warps 5..8   the epilogue
// dy [4096][14336] at rank 64: 35 us (3.4 TB/s), of which 23 are the steps at 5.1 TB/s and the rest
// the start, the cluster's sums and their writing; x [777][11008] at rank 32: 14 us.
constexpr int kLoadWarps = 4;
constexpr int kNarrowThreads = (kLoadWarps + 1 + 4) * 32;
constexpr int kNarrowMaxStages = 8;

struct NarrowParams {
    RowMaps w;            // x [M][K] or dy [M][N]
    CUtensorMap tm_f;
    Common c;
    int64_t K;            // the contraction's length
    int steps;            // 64-wide steps of one CTA
    int stages, f_bytes;  // ring depth, bytes of the factor in a stage
    int tmem_cols;
    const float* scales;  // backward: s
    const float* u_in;    // backward: u [M][R]
    float* u_out;         // forward: [M][R] or null
};

template <typename T, bool FWD>
__global__ void __launch_bounds__(kNarrowThreads) adapters_narrow_kernel(const __grid_constant__ NarrowParams p)
{
    constexpr int f16 = Is16<T>::f16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[kNarrowMaxStages], empty[kNarrowMaxStages], acc_full;
    __shared__ uint32_t tmem_s;
    __shared__ int abort_flag;
    __shared__ float warp_max[2][4];
    __shared__ int toks[kTileL];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int z = gridDim.x, rank = blockIdx.x;  // the cluster spans the grid's x
    const int stage_bytes = 2 * (int)kAtom + p.f_bytes;
    const Common& c = p.c;

    if (tid == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&acc_full, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    pdl_wait_prior_grids();
    const int t = blockIdx.y;
    if (t >= c.plan.head[3])
        return;  // the whole cluster
    const AdapterTile d = c.plan.tiles_l[t];
    const int rows = 128 / z, row0 = rank * rows;
    if (d.adapter >= c.L) {  // tokens without an adapter: u is zero, nothing reads their slots
        if (FWD && p.u_out)
            for (int i = tid; i < rows * c.R; i += kNarrowThreads)
                if (row0 + i / c.R < d.count)
                    p.u_out[(size_t)c.plan.perm[d.start + row0 + i / c.R] * c.R + i % c.R] = 0.f;
        return;
    }
    if (warp == kLoadWarps)
        tmem_alloc(&tmem_s, (uint32_t)p.tmem_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // only now: a CTA of the next kernel must not take tensor memory that this grid still waits for
    pdl_launch_dependents();
    const uint32_t tmem = tmem_s;
    const int nk = (int)((p.K + 63) / 64);
    const int k_first = rank * p.steps;
    const int n_st = nk - k_first < 0 ? 0 : nk - k_first < p.steps ? nk - k_first : p.steps;
    auto X = [&](int s) { return smem + s * stage_bytes; };
    auto F = [&](int s) { return smem + s * stage_bytes + 2 * kAtom; };
    const int pitch = c.Rq + 4;  // floats: an odd number of 16-byte units, so rows meet all banks

    if (warp < kLoadWarps) {
        const int piece = 8 * warp + lane;  // lanes 0..7: four rows each of a gathered tile
        const bool box = d.first >= 0;
        const int4 tok = box || lane >= 8 ? make_int4(0, 0, 0, 0) : row_tokens(c.plan, d.start, d.count, piece);
        int it = 0;
        for (; it < n_st; ++it) {
            const int slot = it % p.stages;
            const bool ok = it < p.stages || mbar_wait_bounded(&empty[slot], ((it / p.stages) & 1) ^ 1, c.status);
            if (__any_sync(0xffffffffu, !ok || aborted(&abort_flag))) {
                abort_flag = 1;
                break;
            }
            const int k = (k_first + it) * 64;
            if (lane == 0) {
                if (warp == 0) {
                    mbar_arrive_expect_tx(&full[slot], (unsigned)stage_bytes);
                    tma_load_3d(F(slot), &p.tm_f, FWD ? k : 0, FWD ? 0 : k, d.adapter, &full[slot]);
                } else if (warp == 3) {
                    if (!FWD && c.Rq > 64)
                        tma_load_3d(F(slot) + kAtom, &p.tm_f, 64, k, d.adapter, &full[slot]);
                } else if (box) {
                    load_box(smem_u32(X(slot)) + (warp - 1) * kAtom, &p.w.box, k, d.first + 64 * (warp - 1), &full[slot]);
                }
            }
            __syncwarp();
            if (!box && lane < 8)
                tma_gather4(smem_u32(X(slot)) + piece * 512, &p.w.row, k, tok, &full[slot]);
        }
        for (int j = it - p.stages < 0 ? 0 : it - p.stages; j < it; ++j)  // no copy may land after the exit
            mbar_wait_bounded(&full[j % p.stages], (j / p.stages) & 1, c.status);
    } else if (warp == kLoadWarps) {
        if (lane == 0) {
            const uint32_t ty = f16 ? 0u : (1u << 7) | (1u << 10);
            const uint32_t idesc = (1u << 4) | ty | (FWD ? 0u : 1u << 16) | ((uint32_t)(c.Rq >> 3) << 17) |
                                   ((uint32_t)(128 >> 4) << 24);
            bool ok = true;
            for (int it = 0; it < n_st && ok; ++it) {
                const int slot = it % p.stages;
                ok = mbar_wait_bounded(&full[slot], (it / p.stages) & 1, c.status);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t a = smem_u32(X(slot)), b = smem_u32(F(slot));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    tc_mma<false>(tmem, umma_desc_sw128(a + kk * 32),
                                  FWD ? umma_desc_sw128(b + kk * 32) : umma_desc_sw128_mn(b + kk * 2048, kAtom), idesc,
                                  (it | kk) != 0 ? 1u : 0u);
                tc_commit(&empty[slot]);
            }
            if (!ok)
                abort_flag = 1;
            tc_commit(&acc_full);  // after the last MMA issued, also when stopping early
            mbar_wait_bounded(&acc_full, 0, c.status);
        }
        __syncwarp();
    } else {
        const int q = warp & 3;
        // during the products: the tokens of this CTA's rows, and (backward) its rows of u
        for (int i = tid - (kLoadWarps + 1) * 32; i < rows; i += 128)
            toks[i] = row0 + i < d.count ? c.plan.perm[d.start + row0 + i] : -1;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if constexpr (!FWD) {
            const int per = c.Rq / 4;
            const size_t lo_at = (size_t)c.slots * c.Rq;
            float umax = 0.f;
            for (int i = tid - (kLoadWarps + 1) * 32; i < rows * per; i += 128) {
                const int row = i / per, col = 4 * (i % per);
                const size_t at = ((size_t)t * kTileL + row0 + row) * c.Rq + col;
                float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
                if (toks[row] >= 0 && col < c.R)
                    u = __ldg(reinterpret_cast<const float4*>(p.u_in + (size_t)toks[row] * c.R + col));
                if constexpr (f16) {
                    umax = fmaxf(umax, fmaxf(fmaxf(finite_abs(u.x), finite_abs(u.y)), fmaxf(finite_abs(u.z), finite_abs(u.w))));
                } else {
                    uint2 hi, lo;
                    split2<T>(u.x, u.y, hi.x, lo.x);
                    split2<T>(u.z, u.w, hi.y, lo.y);
                    *reinterpret_cast<uint2*>(c.u_halves + at) = hi;
                    *reinterpret_cast<uint2*>(c.u_halves + lo_at + at) = lo;
                }
            }
            if constexpr (f16) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    umax = fmaxf(umax, __shfl_xor_sync(0xffffffffu, umax, o));
                if (lane == 0)
                    warp_max[1][warp - kLoadWarps - 1] = umax;
            }
        }
        // this CTA's sums, [128][Rq], into the ring's memory (every MMA, so every copy, is done)
        const bool sums = n_st > 0 && mbar_wait_bounded(&acc_full, 0, c.status) && !aborted(&abort_flag);
        tc_fence_after();
        float* red = reinterpret_cast<float*>(smem) + (size_t)(32 * q + lane) * pitch;
        for (int col = 0; col < c.Rq; col += 16) {
            uint32_t r[16];
            if (sums) {
                tmem_ld16(tmem + (uint32_t)col + ((uint32_t)(32 * q) << 16), r);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    r[j] = 0u;
            }
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                *reinterpret_cast<uint4*>(red + col + j) = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
        }
        tc_fence_before();
    }
    __syncthreads();
    if (z > 1)
        cluster_sync();
    if (warp > kLoadWarps) {
        // a power of two of lanes takes a row, four columns a lane: 32 / lanes rows a warp at a time
        const float sc = FWD ? 1.f : p.scales[d.adapter];
        const uint32_t mine = smem_u32(smem);
        const int lanes = c.Rq <= 16 ? 4 : c.Rq <= 32 ? 8 : c.Rq <= 64 ? 16 : 32, at_once = 4 * (32 / lanes);
        const int col = 4 * (lane & (lanes - 1));
        const size_t lo_at = (size_t)c.slots * c.Rq;
        float vmax = 0.f;
        for (int r0 = 0; r0 < rows; r0 += at_once) {
            const int row = row0 + r0 + (warp - kLoadWarps - 1) * (32 / lanes) + lane / lanes;
            const bool mine_ok = row < row0 + rows, in = mine_ok && row < d.count && col < c.R;
            const size_t at = ((size_t)t * kTileL + row) * c.Rq + col;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in) {
                const uint32_t from = mine + (uint32_t)(row * pitch + col) * 4u;
                float4 v[kMaxSplit];
#pragma unroll
                for (int j = 0; j < kMaxSplit; ++j)
                    v[j] = j < z ? ld_peer_v4(peer_smem(from, (uint32_t)j)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int j = 0; j < kMaxSplit; ++j) {
                    s.x += v[j].x;
                    s.y += v[j].y;
                    s.z += v[j].z;
                    s.w += v[j].w;
                }
                s = make_float4(sc * s.x, sc * s.y, sc * s.z, sc * s.w);
                if (FWD && p.u_out)
                    *reinterpret_cast<float4*>(p.u_out + (size_t)toks[row - row0] * c.R + col) = s;
            }
            float to = 1.f, back = 1.f;
            if constexpr (f16) {
                float top = fmaxf(fmaxf(finite_abs(s.x), finite_abs(s.y)), fmaxf(finite_abs(s.z), finite_abs(s.w)));
                vmax = fmaxf(vmax, top);
                for (int o = lanes >> 1; o > 0; o >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                half_scale<T>(top, to, back);
                if (col == 0 && mine_ok)
                    c.row_back[(size_t)t * kTileL + row] = back;
            }
            if (mine_ok && col < c.Rq) {
                uint2 hi, lo;
                split2<T>(s.x * to, s.y * to, hi.x, lo.x);
                split2<T>(s.z * to, s.w * to, hi.y, lo.y);
                *reinterpret_cast<uint2*>(c.row_halves + at) = hi;
                *reinterpret_cast<uint2*>(c.row_halves + lo_at + at) = lo;
                if constexpr (!FWD && f16)
                    *reinterpret_cast<float4*>(c.v + at) = s;
            }
        }
        if constexpr (!FWD && f16) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, o));
            if (lane == 0)
                warp_max[0][warp - kLoadWarps - 1] = vmax;
            asm volatile("bar.sync 1, 128;" ::: "memory");
            const int which = tid - (kLoadWarps + 1) * 32;
            if (which < 2) {
                const float* w = warp_max[which];
                c.tile_max[((size_t)t * kMaxSplit + rank) * 2 + which] = fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3]));
            }
        }
    }
    if (z > 1)
        cluster_sync();  // no CTA's shared memory goes while another reads it
    else
        __syncthreads();
    if (warp == kLoadWarps)
        tmem_dealloc(tmem, (uint32_t)p.tmem_cols);
}

// The grams' halves for fp16, scaled by the adapter's power of two: a CTA for each tile.
struct SplitParams {
    Common c;
    const float* u;  // [M][R]
    int parts;       // CTAs of a tile in the narrow kernel: maxima of a tile
};

QLIN_DEV float adapter_max(const Common& c, int i, int which, int parts, int lane)
{
    float top = 0.f;
    const int t0 = c.plan.tile_l0[i], n = (c.plan.tile_l0[i + 1] - t0) * parts;
    for (int e = lane; e < n; e += 32)
        top = fmaxf(top, c.tile_max[((size_t)(t0 + e / parts) * kMaxSplit + e % parts) * 2 + which]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    return top;
}

__global__ void __launch_bounds__(256) adapters_split_kernel(const SplitParams p)
{
    const Common& c = p.c;
    pdl_launch_dependents();
    pdl_wait_prior_grids();
    const int t = blockIdx.x, lane = threadIdx.x & 31;
    if (t >= c.plan.head[5])
        return;
    const AdapterTile d = c.plan.tiles_l[t];
    float tov, tou, back;
    half_scale<__half>(adapter_max(c, d.adapter, 0, p.parts, lane), tov, back);
    half_scale<__half>(adapter_max(c, d.adapter, 1, p.parts, lane), tou, back);
    const int per = c.Rq / 4;
    const size_t lo_at = (size_t)c.slots * c.Rq;
    for (int i = threadIdx.x; i < kTileL * per; i += 256) {
        const int row = i / per, col = 4 * (i % per);
        const size_t at = ((size_t)t * kTileL + row) * c.Rq + col;
        const float4 v = __ldcg(reinterpret_cast<const float4*>(c.v + at));
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row < d.count && col < c.R)
            u = __ldg(reinterpret_cast<const float4*>(p.u + (size_t)c.plan.perm[d.start + row] * c.R + col));
        uint2 hi, lo;
        split2<__half>(v.x * tov, v.y * tov, hi.x, lo.x);
        split2<__half>(v.z * tov, v.w * tov, hi.y, lo.y);
        *reinterpret_cast<uint2*>(c.v_halves + at) = hi;
        *reinterpret_cast<uint2*>(c.v_halves + lo_at + at) = lo;
        split2<__half>(u.x * tou, u.y * tou, hi.x, lo.x);
        split2<__half>(u.z * tou, u.w * tou, hi.y, lo.y);
        *reinterpret_cast<uint2*>(c.u_halves + at) = hi;
        *reinterpret_cast<uint2*>(c.u_halves + lo_at + at) = lo;
    }
}

// ------------------------------------------------------------------------------------ wide

// out = base + h F, persistent: the (tile, block of 128 columns) units of the batch, tile by tile, in
// equal contiguous shares, one CTA an SM.  A share is one to a few segments, each of one tile.
//   warps 0..3   the loads: for a segment the halves of h; each block's factor -- forward B_i
//                [128 n][R], K-major; backward A_i [Rq r][128 k], MN-major -- and base [128][128]
//   warp 4       two accumulators of 128 columns; hi and lo halves on the same factor block
//   warps 5..12  32 rows by 64 columns each: the sum, scaled, onto base in shared memory, then out in
//                whole 128-byte pieces of a row (base's own place serves as the staging buffer)
// Tiles of tokens without an adapter pass through without a product (their rows are copied as they
// are), or are left out when out is base itself.
// 4096 tokens by 14336 columns at rank 64: 48 us for 235 MB, 4.9 TB/s, 0.75 of the copy rate.
constexpr int kWideEpi = 8;
constexpr int kWideThreads = (kLoadWarps + 1 + kWideEpi) * 32;
constexpr int kWideMaxStages = 4;
constexpr int kWideCols = 128;

struct WideParams {
    RowMaps base;
    CUtensorMap tm_f, tm_h;
    Common c;
    const float* scales;  // forward
    const void* base_p;   // null: zeros
    void* out;
    int64_t N;
    int blocks;           // of a row
    int stages, f_bytes;
};

template <typename T, bool FWD>
__global__ void __launch_bounds__(kWideThreads, 1) adapters_wide_kernel(const __grid_constant__ WideParams p)
{
    constexpr int f16 = Is16<T>::f16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[kWideMaxStages], empty[kWideMaxStages], acc_full[2], acc_empty[2], h_full, h_empty;
    __shared__ uint32_t tmem_s;
    __shared__ int abort_flag;
    const Common& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1 + kWideEpi);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], kWideEpi);
        }
        mbar_init(&h_full, 1);
        mbar_init(&h_empty, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kLoadWarps)
        tmem_alloc(&tmem_s, 2 * kWideCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();  // after the allocation, as in the narrow kernel
    pdl_wait_prior_grids();
    const uint32_t tmem = tmem_s;
    const int atoms = (c.Rq + 63) / 64, h_half = atoms * 2 * (int)kAtom;
    constexpr int base_bytes = 4 * (int)kAtom;
    const int stage_bytes = base_bytes + p.f_bytes;
    uint8_t* Hs = smem;  // hi, then lo: [atoms][128 rows][128 bytes]
    auto B = [&](int s) { return smem + 2 * h_half + s * stage_bytes; };
    auto F = [&](int s) { return smem + 2 * h_half + s * stage_bytes + base_bytes; };
    // this CTA's units; tiles of tokens without an adapter come last and count where they are copied
    const int64_t units = (int64_t)c.plan.head[p.base_p == p.out ? 5 : 3] * p.blocks;
    const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
    // blocks b0 .. b1 - 1 of the tile that unit u belongs to
    auto segment = [&](int64_t u, int& t, int& b0, int& b1) {
        t = (int)(u / p.blocks);
        b0 = (int)(u - (int64_t)t * p.blocks);
        b1 = (int)(u1 - u < p.blocks - b0 ? b0 + (u1 - u) : p.blocks);
    };

    if (warp < kLoadWarps) {
        const int piece = 16 * (warp & 1) + (lane & 15);  // lanes 0..15: four rows each of a gathered 64-column half
        int it = 0, seg = 0;
        bool ok = true;
        for (int64_t u = u0; u < u1 && ok;) {
            int t, b0, b1;
            segment(u, t, b0, b1);
            u += b1 - b0;
            const AdapterTile d = c.plan.tiles_l[t];
            const bool none = d.adapter >= c.L;
            const bool box = d.first >= 0;
            const int4 tok = box ? make_int4(0, 0, 0, 0) : row_tokens(c.plan, d.start, d.count, piece);
            if (warp == 0 && !none) {  // h of the segment, once the MMAs of the last one are done
                if (seg > 0 && !mbar_wait_bounded(&h_empty, (seg & 1) ^ 1, c.status))
                    ok = false;
                if (ok && lane == 0) {
                    mbar_arrive_expect_tx(&h_full, 2u * (unsigned)h_half);
                    for (int half = 0; half < 2; ++half)
                        for (int a = 0; a < atoms; ++a)
                            tma_load_2d(Hs + half * h_half + a * 2 * kAtom, &p.tm_h, a * 64,
                                        (int)(half * c.slots) + t * kTileL, &h_full);
                }
                ++seg;
            }
            for (int b = b0; b < b1 && ok; ++b, ++it) {
                const int slot = it % p.stages;
                ok = it < p.stages || mbar_wait_bounded(&empty[slot], ((it / p.stages) & 1) ^ 1, c.status);
                ok = __all_sync(0xffffffffu, ok && !aborted(&abort_flag));
                if (!ok)
                    break;
                const int n = b * kWideCols;
                if (lane == 0) {
                    if (warp == 0)
                        mbar_arrive_expect_tx(&full[slot], (unsigned)((none ? 0 : p.f_bytes) + (p.base_p ? base_bytes : 0)));
                    if (box && p.base_p)  // a quarter of base: 64 columns by 64 rows
                        load_box(smem_u32(B(slot)) + warp * kAtom, &p.base.box, n + (warp >> 1) * 64, d.first + (warp & 1) * 64,
                                 &full[slot]);
                    if (!none && warp < (FWD ? atoms : 2)) {
                        if constexpr (FWD)
                            tma_load_3d(F(slot) + warp * 2 * kAtom, &p.tm_f, warp * 64, n, d.adapter, &full[slot]);
                        else
                            tma_load_3d(F(slot) + warp * c.Rq * 128, &p.tm_f, n + warp * 64, 0, d.adapter, &full[slot]);
                    }
                }
                __syncwarp();
                if (!box && p.base_p && lane < 16) {
                    const int a = warp >> 1;
                    tma_gather4(smem_u32(B(slot)) + a * 2 * kAtom + piece * 512, &p.base.row, n + a * 64, tok, &full[slot]);
                }
            }
        }
        if (!ok)
            abort_flag = 1;
        if (warp == 0) {  // no copy may land after the exit
            if (seg > 0)
                mbar_wait_bounded(&h_full, (seg - 1) & 1, c.status);
            for (int j = it - p.stages < 0 ? 0 : it - p.stages; j < it; ++j)
                mbar_wait_bounded(&full[j % p.stages], (j / p.stages) & 1, c.status);
        }
    } else if (warp == kLoadWarps) {
        if (lane == 0) {
            const uint32_t ty = f16 ? 0u : (1u << 7) | (1u << 10);
            const uint32_t idesc = (1u << 4) | ty | (FWD ? 0u : 1u << 16) | ((uint32_t)(kWideCols >> 3) << 17) |
                                   ((uint32_t)(128 >> 4) << 24);
            bool ok = true;
            int it = 0, seg = 0, last = -1;
            for (int64_t u = u0; u < u1 && ok;) {
                int t, b0, b1;
                segment(u, t, b0, b1);
                u += b1 - b0;
                const bool none = c.plan.tiles_l[t].adapter >= c.L;
                ok = none || mbar_wait_bounded(&h_full, seg & 1, c.status);
                for (int b = b0; b < b1 && ok; ++b, ++it) {
                    const int slot = it % p.stages, buf = it & 1;
                    ok = mbar_wait_bounded(&acc_empty[buf], ((it >> 1) & 1) ^ 1, c.status) &&
                         mbar_wait_bounded(&full[slot], (it / p.stages) & 1, c.status);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint32_t h = smem_u32(Hs), f = smem_u32(F(slot));
                    for (int kk = 0; kk < (none ? 0 : c.Rq / 16); ++kk) {
                        const uint64_t fd = FWD ? umma_desc_sw128(f + (kk >> 2) * 2 * kAtom + (kk & 3) * 32)
                                                : umma_desc_sw128_mn(f + kk * 2048, (uint32_t)(c.Rq * 128));
#pragma unroll
                        for (int half = 0; half < 2; ++half)
                            tc_mma<false>(tmem + (uint32_t)(buf * kWideCols),
                                          umma_desc_sw128(h + half * h_half + (kk >> 2) * 2 * kAtom + (kk & 3) * 32), fd,
                                          idesc, (kk | half) != 0 ? 1u : 0u);
                    }
                    tc_commit(&empty[slot]);
                    tc_commit(&acc_full[buf]);
                    last = it;
                }
                if (!none) {
                    tc_commit(&h_empty);
                    ++seg;
                }
            }
            if (!ok)
                abort_flag = 1;
            if (last >= 0)  // every MMA issued has completed before TMEM is released
                mbar_wait_bounded(&acc_full[last & 1], (last >> 1) & 1, c.status);
        }
        __syncwarp();
    } else {
        const int w = warp - kLoadWarps - 1, q = warp & 3, half = w >> 2, row = 32 * q + lane;
        T* out = static_cast<T*>(p.out);
        int it = 0;
        bool ok = true;
        for (int64_t u = u0; u < u1 && ok;) {
            int t, b0, b1;
            segment(u, t, b0, b1);
            u += b1 - b0;
            const AdapterTile d = c.plan.tiles_l[t];
            const bool none = d.adapter >= c.L;
            const int my_tok = row < d.count ? c.plan.perm[d.start + row] : -1;
            float rs = FWD && !none ? p.scales[d.adapter] : 1.f;
            if constexpr (f16)
                rs *= none ? 1.f : __ldcg(c.row_back + (size_t)t * kTileL + row);
            for (int b = b0; b < b1; ++b, ++it) {
                const int slot = it % p.stages, buf = it & 1;
                if (!mbar_wait_bounded(&full[slot], (it / p.stages) & 1, c.status) ||
                    !mbar_wait_bounded(&acc_full[buf], (it >> 1) & 1, c.status) || aborted(&abort_flag)) {
                    abort_flag = 1;
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t acc = tmem + (uint32_t)(buf * kWideCols + half * 64) + ((uint32_t)(32 * q) << 16);
                uint8_t* at = B(slot) + half * 2 * kAtom;
                uint32_t r[4][16];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    tmem_ld16_nowait(acc + 16u * e, r[e]);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&acc_empty[buf]);
#pragma unroll
                for (int un = 0; un < 8; ++un) {
                    uint4* bp = reinterpret_cast<uint4*>(at + swz128(row, un));
                    const uint4 bv = p.base_p ? *bp : make_uint4(0u, 0u, 0u, 0u);
                    if (none) {
                        if (!p.base_p)
                            *bp = bv;
                        continue;
                    }
                    const uint32_t bw[4] = {bv.x, bv.y, bv.z, bv.w};
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[e] = pack_h16x2(
                            fmaf(__uint_as_float(r[un >> 1][(un & 1) * 8 + 2 * e]), rs, h16_to_float(bw[e], f16)),
                            fmaf(__uint_as_float(r[un >> 1][(un & 1) * 8 + 2 * e + 1]), rs, h16_to_float(bw[e] >> 16, f16)),
                            f16);
                    *bp = make_uint4(o[0], o[1], o[2], o[3]);
                }
                __syncwarp();
                const int64_t n = (int64_t)b * kWideCols + half * 64 + 8 * (lane & 7);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int rr = 4 * e + (lane >> 3);
                    const int tok = __shfl_sync(0xffffffffu, my_tok, rr);
                    const uint4 v = *reinterpret_cast<const uint4*>(at + swz128(32 * q + rr, lane & 7));
                    if (tok >= 0 && n < p.N)
                        *reinterpret_cast<uint4*>(out + (size_t)tok * p.N + n) = v;
                }
                fence_proxy_async_smem();  // the next copy into this place comes after these accesses
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&empty[slot]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kLoadWarps)
        tmem_dealloc(tmem, 2 * kWideCols);
}

// ------------------------------------------------------------------------------------ decode

// Both products in one launch, for few tokens: a cluster for each tile of 8 tokens of one adapter.
// Latency bounds it (one token of a 4096 x 4096 layer at rank 16 reads 0.26 MB), so everything a
// warp needs is requested at once, straight into MMA fragments: ranks are the MMA's 16 rows, tokens
// its 8 columns, and the contraction index is permuted so that a fragment is 16 contiguous bytes of
// a row of A_i or x.  The CTAs split the contraction; each sends its sums [Rq][8] to every CTA of
// the cluster (one barrier), and takes its share of the 128-column blocks of the second product,
// whose factor it has prefetched into L2 meanwhile.
// 1 token, 4096 x 4096, rank 16: 4.1 us (narrow and wide: 10.2); 61 tokens of 32 adapters, 4096 ->
// 11008: 8.1 us for 23 MB.
constexpr int kDecodeWarps = 8;

struct DecodeParams {
    Common c;
    const void* x;
    const void* a;
    const void* b;
    const float* scales;
    const void* base;
    void* out;
    float* u;
    int64_t K, N;
};

QLIN_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
QLIN_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
QLIN_DEV void st_peer(uint32_t addr, float v) { asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory"); }

template <typename T>
QLIN_DEV void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (Is16<T>::f16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        mma_bf16_16816(d, a, b0, b1);
}

template <typename T, int KT>
__global__ void __launch_bounds__(kDecodeWarps * 32) adapters_decode_kernel(const DecodeParams p)
{
    constexpr int f16 = Is16<T>::f16, RQ = 16 * KT, kUnroll = KT <= 2 ? 4 : KT == 4 ? 2 : 1;
    extern __shared__ __align__(16) float sm[];
    const Common& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, j = lane >> 2, q4 = lane & 3;
    const int z = gridDim.x, rank = blockIdx.x;
    float* red = sm;                            // [warps][RQ][8]
    float* recv = red + kDecodeWarps * RQ * 8;  // [z][RQ][8]
    float* us = recv + z * RQ * 8;              // [8][RQ + 4]
    pdl_launch_dependents();
    pdl_wait_prior_grids();
    const int t = blockIdx.y;
    if (t >= c.plan.head[2])
        return;  // the whole cluster
    const AdapterTile d = c.plan.tiles_s[t];
    const T* base = static_cast<const T*>(p.base);
    T* out = static_cast<T*>(p.out);
    const int blocks_n = (int)((p.N + 127) / 128);
    if (d.adapter >= c.L) {
        const int vecs = (int)(p.N / 8);
        if (base != out)
            for (int i = rank * 256 + tid; i < d.count * vecs; i += z * 256) {
                const size_t at = (size_t)c.plan.perm[d.start + i / vecs] * p.N + 8 * (i % vecs);
                *reinterpret_cast<uint4*>(out + at) =
                    base ? *reinterpret_cast<const uint4*>(base + at) : make_uint4(0u, 0u, 0u, 0u);
            }
        if (p.u && rank == 0)
            for (int i = tid; i < d.count * c.R; i += 256)
                p.u[(size_t)c.plan.perm[d.start + i / c.R] * c.R + i % c.R] = 0.f;
        return;
    }
    cluster_arrive();  // every CTA of the cluster has started before one writes to another
    const T* fb = static_cast<const T*>(p.b) + (size_t)d.adapter * p.N * c.R;
    {
        // this CTA's blocks of the second factor: 128 R elements each, every z-th block
        const int lines = 128 * c.R * (int)sizeof(T) / 128;
        const char* end = reinterpret_cast<const char*>(fb + (size_t)p.N * c.R);
        const int mine = blocks_n > rank ? (blocks_n - 1 - rank) / z + 1 : 0;
        for (int i = tid; i < mine * lines && i < 4 * 256; i += 256) {
            const char* at = reinterpret_cast<const char*>(fb) +
                             ((size_t)(rank + (i / lines) * z) * lines + i % lines) * 128;
            if (at < end)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
        }
    }
    // ---- A_i x: ranks are MMA rows, tokens columns
    const int steps = (int)((p.K + 31) / 32), per = (steps + z - 1) / z;
    const int s1 = min(steps, (rank + 1) * per);
    const T* xr = static_cast<const T*>(p.x);
    const int my_tok = j < d.count ? c.plan.perm[d.start + j] : -1;
    if (my_tok >= 0)
        xr += (size_t)my_tok * p.K;
    const T* fa = static_cast<const T*>(p.a) + (size_t)d.adapter * c.R * p.K;
    float acc[KT][4] = {};
    for (int s = rank * per + warp; s < s1; s += kDecodeWarps * kUnroll) {
        uint4 xv[kUnroll], av[kUnroll][KT][2];
#pragma unroll
        for (int e = 0; e < kUnroll; ++e) {
            const int64_t k = (int64_t)(s + e * kDecodeWarps) * 32 + 8 * q4;
            const bool in = s + e * kDecodeWarps < s1 && k < p.K;
            xv[e] = in && my_tok >= 0 ? ldg_cg_v4(xr + k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int m = 0; m < KT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = 16 * m + j + 8 * h;
                    av[e][m][h] = in && r < c.R ? ldg_stream_v4(fa + (size_t)r * p.K + k) : make_uint4(0u, 0u, 0u, 0u);
                }
        }
#pragma unroll
        for (int e = 0; e < kUnroll; ++e)
#pragma unroll
            for (int m = 0; m < KT; ++m) {
                const uint32_t a0[4] = {av[e][m][0].x, av[e][m][1].x, av[e][m][0].y, av[e][m][1].y};
                const uint32_t a1[4] = {av[e][m][0].z, av[e][m][1].z, av[e][m][0].w, av[e][m][1].w};
                mma_16816<T>(acc[m], a0, xv[e].x, xv[e].y);
                mma_16816<T>(acc[m], a1, xv[e].z, xv[e].w);
            }
    }
#pragma unroll
    for (int m = 0; m < KT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float2*>(red + (warp * RQ + 16 * m + j + 8 * h) * 8 + 2 * q4) =
                make_float2(acc[m][2 * h], acc[m][2 * h + 1]);
    __syncthreads();
    cluster_wait();
    for (int i = tid; i < RQ * 8; i += 256) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kDecodeWarps; ++w)
            sum += red[w * RQ * 8 + i];
        const uint32_t at = smem_u32(recv + rank * RQ * 8 + i);
        for (int k = 0; k < z; ++k)
            st_peer(peer_smem(at, (uint32_t)k), sum);
    }
    cluster_sync();
    for (int i = tid; i < RQ * 8; i += 256) {
        float sum = 0.f;
        for (int k = 0; k < z; ++k)
            sum += recv[k * RQ * 8 + i];
        const int r = i >> 3, tok = i & 7;
        const bool in = tok < d.count && r < c.R;
        us[tok * (RQ + 4) + r] = in ? sum : 0.f;
        if (p.u && rank == 0 && in)
            p.u[(size_t)c.plan.perm[d.start + tok] * c.R + r] = sum;
    }
    __syncthreads();
    // ---- B_i u: columns n are MMA rows (row j of MMA q is column 8 j + q of the block, row j + 8
    // is 64 columns on), tokens columns
    uint32_t hi[KT][2], lo[KT][2];
    float4 v[KT];
    float top = 0.f, to = 1.f, back = 1.f;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
        v[k] = *reinterpret_cast<const float4*>(us + j * (RQ + 4) + 16 * k + 4 * q4);
        top = fmaxf(fmaxf(top, fmaxf(finite_abs(v[k].x), finite_abs(v[k].y))),
                    fmaxf(finite_abs(v[k].z), finite_abs(v[k].w)));
    }
    if constexpr (f16) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        half_scale<T>(top, to, back);
    }
#pragma unroll
    for (int k = 0; k < KT; ++k) {
        split2<T>(v[k].x * to, v[k].y * to, hi[k][0], lo[k][0]);
        split2<T>(v[k].z * to, v[k].w * to, hi[k][1], lo[k][1]);
    }
    const float sc = p.scales[d.adapter];
    float rs[2];
    int tok[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // this thread's two tokens of the sums
        rs[e] = sc * __shfl_sync(0xffffffffu, back, 4 * (2 * q4 + e));
        tok[e] = __shfl_sync(0xffffffffu, my_tok, 4 * (2 * q4 + e));
    }
    for (int blk = rank + z * warp; blk < blocks_n; blk += z * kDecodeWarps) {
        const int64_t nb = (int64_t)blk * 128;
        uint4 bv[2][2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t n = nb + 64 * h + 8 * j;
                bv[e][h] = base && tok[e] >= 0 && n < p.N
                               ? *reinterpret_cast<const uint4*>(base + (size_t)tok[e] * p.N + n)
                               : make_uint4(0u, 0u, 0u, 0u);
            }
        float o[8][4] = {};
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            const bool rin = 16 * k + 4 * q4 < c.R;
            uint2 f[8][2];
#pragma unroll
            for (int q = 0; q < 8; ++q)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t n = nb + 64 * h + 8 * j + q;
                    f[q][h] = rin && n < p.N ? __ldg(reinterpret_cast<const uint2*>(fb + (size_t)n * c.R + 16 * k + 4 * q4))
                                             : make_uint2(0u, 0u);
                }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const uint32_t a[4] = {f[q][0].x, f[q][1].x, f[q][0].y, f[q][1].y};
                mma_16816<T>(o[q], a, hi[k][0], hi[k][1]);
                mma_16816<T>(o[q], a, lo[k][0], lo[k][1]);
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t n = nb + 64 * h + 8 * j;
                if (tok[e] < 0 || n >= p.N)
                    continue;
                const uint32_t bw[4] = {bv[e][h].x, bv[e][h].y, bv[e][h].z, bv[e][h].w};
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    w[q] = pack_h16x2(fmaf(o[2 * q][2 * h + e], rs[e], h16_to_float(bw[q], f16)),
                                      fmaf(o[2 * q + 1][2 * h + e], rs[e], h16_to_float(bw[q] >> 16, f16)), f16);
                *reinterpret_cast<uint4*>(out + (size_t)tok[e] * p.N + n) = make_uint4(w[0], w[1], w[2], w[3]);
            }
    }
}

// ------------------------------------------------------------------------------------ grams

// One cluster for each adapter and strip of 256 columns of dy or x: D = H^T S over the adapter's tokens, 64 at a time, the steps dealt round the cluster's CTAs.  S (dy, x or the
// restored x) and H (the halves of u or v) lie token by token in shared memory, which is MN-major
// for both operands; nothing is transposed.
//   warps 0..3   the loads: S in 64-column boxes or gathers (codes: 128-byte ones), H in 64-rank boxes
//   warp 4       tensor memory, the MMAs (M = 128 ranks, N = 256 columns, K = 16).  Up to rank 64 the
//                128 rows are the 64 of hi and the 64 of lo, added at the end: one MMA a step of 16
//                (columns as M and ranks as N took four, each no faster)
//   warps 5..20  codes: s q in fp32, rounded once to the operand type, into a ring of two buffers;
//                rows past the adapter's last token: zeros (only there, so what another adapter's
//                row holds enters no sum); then the epilogue
// 4096 tokens of 4 adapters, 14336 bf16 columns and 4096 of codes, rank 64: 49 - 56 us by how the
// tokens fall on the adapters, for 135 MB; a step of 48 KB comes at 62 GB/s an SM.
constexpr int kGramWork = 16;
constexpr int kGramThreads = (kLoadWarps + 1 + kGramWork) * 32;
constexpr int kGramMaxStages = 6;
constexpr int kGramPitch = 257;
constexpr int kMaxGramSplit = 8;

struct GramParams {
    RowMaps dy, x;         // x: 16-bit, or the codes
    CUtensorMap tm_u, tm_v;
    Common c;
    const float* scales;
    const float* q_scale;  // [K/g][M]; null: x is not codes
    int g_shift;
    int64_t N, K;
    int strips_y, strips_x;
    void* da;  // [L][R][K]
    void* db;  // [L][N][R]
    int parts;  // CTAs of a tile in the narrow kernel: maxima of a tile
    int tmem_cols, room;  // room: bytes of shared memory for the rings
    int z;                // CTAs of a cluster
};

template <typename T>
__global__ void __launch_bounds__(kGramThreads, 1) adapters_gram_kernel(const __grid_constant__ GramParams p)
{
    constexpr int f16 = Is16<T>::f16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[kGramMaxStages], empty[kGramMaxStages], ready[2], taken[2], acc_full, tail;
    __shared__ uint32_t tmem_s;
    __shared__ int abort_flag;
    const Common& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int z = p.z, rank = blockIdx.x % z, job = blockIdx.x / z;
    pdl_wait_prior_grids();
    const int strips = p.strips_y + p.strips_x;
    const int i = job / strips, strip = job % strips;
    const bool of_dy = strip < p.strips_y, of_q = !of_dy && p.q_scale;
    const int64_t n0 = (int64_t)(of_dy ? strip : strip - p.strips_y) * 256, ncols = of_dy ? p.N : p.K;
    const int seg0 = c.plan.seg[i], tokens = c.plan.seg[i + 1] - seg0, tile0 = c.plan.tile_l0[i];
    if (tokens == 0) {  // the whole cluster: zeros
        const int64_t n = ncols - n0 < 256 ? ncols - n0 : 256;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        if (of_dy) {
            uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(p.db) + ((size_t)i * p.N + n0) * c.R);
            for (int64_t e = rank * kGramThreads + tid; e < n * c.R / 8; e += z * kGramThreads)
                o[e] = zero;
        } else {
            const int vecs = (int)(n / 8);
            for (int e = rank * kGramThreads + tid; e < vecs * c.R; e += z * kGramThreads)
                *reinterpret_cast<uint4*>(static_cast<T*>(p.da) + ((size_t)i * c.R + e / vecs) * p.K + n0 + 8 * (e % vecs)) = zero;
        }
        return;
    }
    if (tid == 0) {
        for (int s = 0; s < kGramMaxStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ready[b], kGramWork / 2);
            mbar_init(&taken[b], 1);
        }
        mbar_init(&acc_full, 1);
        mbar_init(&tail, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kLoadWarps)
        tmem_alloc(&tmem_s, (uint32_t)p.tmem_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_s;
    pdl_launch_dependents();  // after the allocation, as in the narrow kernel
    const int steps = (tokens + 63) / 64;
    const int n_st = steps > rank ? (steps - 1 - rank) / z + 1 : 0;  // steps rank, rank + z, ...
    const bool stacked = c.Rq <= 64;  // hi and lo are the two 64-rank atoms of one operand
    const int h_half = (c.Rq + 63) / 64 * (int)kAtom;
    const int src_bytes = of_q ? 2 * (int)kAtom : 4 * (int)kAtom, stage_bytes = src_bytes + 2 * h_half;
    const int ring = of_q ? 2 * 4 * (int)kAtom : 0;  // decoded buffers, first in shared memory
    const int stages = min(kGramMaxStages, (p.room - ring) / stage_bytes);
    auto S = [&](int s) { return smem + ring + s * stage_bytes; };
    auto H = [&](int s) { return smem + ring + s * stage_bytes + src_bytes; };
    auto D = [&](int b) { return smem + b * 4 * kAtom; };
    auto rows_of = [&](int it) { return min(64, tokens - (rank + it * z) * 64); };
    // a step waits for the worker warps where there is something to decode or to clear
    auto worked = [&](int it) { return of_q || rows_of(it) < 64; };

    if (warp < kLoadWarps) {
        const RowMaps& m = of_dy ? p.dy : p.x;
        const int width = of_q ? 128 : 64, blocks = src_bytes / (int)kAtom;  // 128-byte columns: a warp each
        // a step's tile and tokens are read a step ahead: their latency is longer than a step
        AdapterTile next;
        int4 next_tok;
        auto look = [&](int it) {
            const int step = rank + it * z;
            next = c.plan.tiles_l[tile0 + (step >> 1)];
            next_tok = row_tokens(c.plan, seg0 + step * 64, rows_of(it), lane & 15);
        };
        if (n_st > 0)
            look(0);
        int it = 0;
        for (; it < n_st; ++it) {
            const int slot = it % stages, step = rank + it * z;
            const AdapterTile d = next;
            const int4 tok = next_tok;
            if (it + 1 < n_st)
                look(it + 1);
            const bool ok = it < stages || mbar_wait_bounded(&empty[slot], ((it / stages) & 1) ^ 1, c.status);
            if (__any_sync(0xffffffffu, !ok || aborted(&abort_flag))) {
                abort_flag = 1;
                break;
            }
            const uint32_t s0 = smem_u32(S(slot));
            if (lane == 0) {
                if (warp == 0)
                    mbar_arrive_expect_tx(&full[slot], (unsigned)stage_bytes);
                if (d.first >= 0 && warp < blocks)
                    load_box(s0 + warp * kAtom, &m.box, (int)n0 + warp * width, d.first + (step & 1) * 64, &full[slot]);
                // the atoms of hi, then of lo, from the last warp on
                const int a = kLoadWarps - 1 - warp, atoms = h_half / (int)kAtom, slot0 = (tile0 + (step >> 1)) * kTileL + (step & 1) * 64;
                if (a < 2 * atoms)
                    tma_load_2d(H(slot) + a * kAtom, of_dy ? &p.tm_u : &p.tm_v, a % atoms * 64,
                                (int)(a / atoms * c.slots) + slot0, &full[slot]);
            }
            __syncwarp();
            if (d.first < 0 && warp < blocks && lane < 16)
                tma_gather4(s0 + warp * kAtom + lane * 512, &m.row, (int)n0 + warp * width, tok, &full[slot]);
        }
        for (int j = it - stages < 0 ? 0 : it - stages; j < it; ++j)
            mbar_wait_bounded(&full[j % stages], (j / stages) & 1, c.status);
    } else if (warp == kLoadWarps) {
        if (lane == 0) {
            const uint32_t ty = f16 ? 0u : (1u << 7) | (1u << 10);
            const uint32_t idesc =
                (1u << 4) | ty | (1u << 15) | (1u << 16) | ((uint32_t)(256 >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
            const int halves = stacked ? 1 : 2;
            bool ok = true;
            for (int it = 0; it < n_st && ok; ++it) {
                const int slot = it % stages, b = it & 1;
                ok = mbar_wait_bounded(&full[slot], (it / stages) & 1, c.status);
                if (ok && worked(it)) {
                    // without codes there is one such step, the last: it has landed, the workers clear it
                    if (!of_q)
                        mbar_arrive(&tail);
                    ok = mbar_wait_bounded(&ready[of_q ? b : 0], of_q ? (it >> 1) & 1 : 0, c.status);
                }
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t a = smem_u32(of_q ? D(b) : S(slot)), h = smem_u32(H(slot));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    for (int half = 0; half < halves; ++half)
                        tc_mma<false>(tmem, umma_desc_sw128_mn(h + half * h_half + kk * 2048, kAtom),
                                      umma_desc_sw128_mn(a + kk * 2048, kAtom), idesc, (it | kk | half) != 0 ? 1u : 0u);
                tc_commit(&empty[slot]);
                if (of_q)
                    tc_commit(&taken[b]);
            }
            if (!ok)
                abort_flag = 1;
            tc_commit(&acc_full);
            mbar_wait_bounded(&acc_full, 0, c.status);
        }
        __syncwarp();
    } else {
        const int w = warp - kLoadWarps - 1;
        bool ok = true;
        if (of_q) {
            // warps 0 - 7 take the even steps, 8 - 15 the odd ones; 64-column atom w & 3, rows 32 (w & 4) / 4
            // .. +31: four chunks of 16 codes a thread; the rows of a phase (r and r + 4) meet no bank
            // twice, loading or storing
            const int odd = w >> 3, atom = w & 3, row0 = (w >> 2 & 1) * 32 + (lane >> 3) + ((lane >> 2) & 1) * 4;
            const int unit = (atom & 1) * 4 + (lane & 3), bunit = 2 * (lane & 3), swap = (lane >> 2) & 1;
            const int64_t k = n0 + atom * 64;
            const float* sc = k < p.K ? p.q_scale + (k >> p.g_shift) * c.M : nullptr;
            // a step's tokens are read two of this warp's steps ahead, their scales one
            float next[4];
            int tok[4];
            auto load_tokens = [&](int it) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = row0 + 8 * e;
                    tok[e] = it < n_st && sc && row < rows_of(it) ? c.plan.perm[seg0 + (rank + it * z) * 64 + row] : -1;
                }
            };
            auto load_scales = [&]() {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    next[e] = tok[e] >= 0 ? __ldg(sc + tok[e]) : 0.f;
            };
            load_tokens(odd);
            load_scales();
            load_tokens(odd + 2);
            for (int it = odd; it < n_st; it += 2) {
                float s[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[e] = next[e];
                load_scales();
                load_tokens(it + 4);
                const int slot = it % stages, b = it & 1;
                // first the buffer: the MMAs of step it - 2, and so those of the slot's last use, are done,
                // and full can only be in the phase that this step ends (a group sees every other one)
                if ((it >= 2 && !mbar_wait_bounded(&taken[b], ((it >> 1) & 1) ^ 1, c.status)) ||
                    !mbar_wait_bounded(&full[slot], (it / stages) & 1, c.status) || aborted(&abort_flag)) {
                    ok = false;
                    break;
                }
                const uint8_t* raw = S(slot) + (atom >> 1) * kAtom;
                const uint32_t dst = smem_u32(D(b)) + atom * kAtom;
                uint4 v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = *reinterpret_cast<const uint4*>(raw + swz128(row0 + 8 * e, unit));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t cw[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
                    uint32_t o[8];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint32_t u = cw[y] ^ 0x80808080u;
                        float fv[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x)  // the byte in the mantissa of 2^23: exact
                            fv[x] = (__uint_as_float(prmt(u, 0x4B000000u, 0x7650u + (uint32_t)x)) - 8388736.f) * s[e];
                        o[2 * y] = pack_h16x2(fv[0], fv[1], f16);
                        o[2 * y + 1] = pack_h16x2(fv[2], fv[3], f16);
                    }
                    const int row = row0 + 8 * e;
                    const uint32_t lo = dst + swz128(row, bunit), hi = dst + swz128(row, bunit + 1);
                    if (swap) {
                        st_shared_v4(hi, o[4], o[5], o[6], o[7]);
                        st_shared_v4(lo, o[0], o[1], o[2], o[3]);
                    } else {
                        st_shared_v4(lo, o[0], o[1], o[2], o[3]);
                        st_shared_v4(hi, o[4], o[5], o[6], o[7]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&ready[b]);
            }
        } else if (n_st > 0 && rows_of(n_st - 1) < 64) {
            // the adapter's last step: zeros past its last token
            const int it = n_st - 1, slot = it % stages, r0 = rows_of(it);
            // told by the MMA thread, which follows every phase of the ring (a wait for one phase of full
            // alone would take an earlier one of the same parity for it)
            ok = mbar_wait_bounded(&tail, 0, c.status);
            if (ok) {
                const uint32_t s0 = smem_u32(S(slot));
                for (int e = w * 32 + lane; e < (64 - r0) * 32 && w < kGramWork / 2; e += kGramWork * 16)
                    st_shared_v4(s0 + ((e & 31) >> 3) * kAtom + (r0 + (e >> 5)) * 128 + (e & 7) * 16, 0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (ok && lane == 0 && w < kGramWork / 2)
                mbar_arrive(&ready[0]);
        }
        if (!ok)
            abort_flag = 1;
        const bool sums = n_st > 0 && mbar_wait_bounded(&acc_full, 0, c.status) && !aborted(&abort_flag);
        tc_fence_after();
        asm volatile("bar.sync 1, %0;" ::"n"(kGramWork * 32) : "memory");
        // the sums, [128][256] at a pitch of 257: lanes store rows and read columns without conflicts
        const int q = warp & 3, row = 32 * q + lane;
        float* red = reinterpret_cast<float*>(smem) + row * kGramPitch;
        const bool used = (stacked ? row & 63 : row) < c.R;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int col = 64 * (w >> 2) + 16 * e;
            uint32_t r[16];
            if (sums) {
                tmem_ld16(tmem + (uint32_t)col + ((uint32_t)(32 * q) << 16), r);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    r[j] = 0u;
            }
            if (used)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    red[col + j] = __uint_as_float(r[j]);
        }
        tc_fence_before();
    }
    __syncthreads();
    if (z > 1)
        cluster_sync();
    if (warp > kLoadWarps) {
        // CTA j adds the cluster's parts of its share of the 256 columns, in order
        const int share = 256 / z, row0 = rank * share;
        float to, back = 1.f;
        if constexpr (f16)
            half_scale<T>(adapter_max(c, i, of_dy ? 1 : 0, p.parts, lane), to, back);
        const float sc = of_dy ? p.scales[i] * back : back;
        T* da = static_cast<T*>(p.da);
        T* db = static_cast<T*>(p.db);
        const int per = c.R / 4, items = share * per;
        // item e: four ranks of a column; consecutive threads write consecutive elements, ranks of dB's
        // rows (8 bytes a thread), columns of dA's (2 bytes, four rows)
        int row = of_dy ? (tid - (kLoadWarps + 1) * 32) / per : (tid - (kLoadWarps + 1) * 32) % share;
        int r4 = of_dy ? (tid - (kLoadWarps + 1) * 32) % per : (tid - (kLoadWarps + 1) * 32) / share;
        const int step_row = of_dy ? kGramWork * 32 / per : 0, step_r4 = of_dy ? kGramWork * 32 % per : kGramWork * 32 / share;
#pragma unroll 2
        for (int e = tid - (kLoadWarps + 1) * 32; e < items; e += kGramWork * 32) {
            const int64_t n = n0 + row0 + row;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (n < ncols && tokens > 0) {
                const float* red = reinterpret_cast<const float*>(smem) + 4 * r4 * kGramPitch + row0 + row;
                float t[4] = {0.f, 0.f, 0.f, 0.f};
                if (z == 1) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        t[j] = red[j * kGramPitch] + (stacked ? red[(64 + j) * kGramPitch] : 0.f);
                } else {
                    const uint32_t from = smem_u32(red);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float part[kMaxGramSplit], more[kMaxGramSplit];
#pragma unroll
                        for (int k = 0; k < kMaxGramSplit; ++k) {
                            const uint32_t at = peer_smem(from + j * kGramPitch * 4u, (uint32_t)(k < z ? k : 0));
                            part[k] = k < z ? ld_peer(at) : 0.f;
                            more[k] = k < z && stacked ? ld_peer(at + 64 * kGramPitch * 4u) : 0.f;
                        }
#pragma unroll
                        for (int k = 0; k < kMaxGramSplit; ++k)
                            t[j] += part[k] + more[k];
                    }
                }
                s = make_float4(t[0] * sc, t[1] * sc, t[2] * sc, t[3] * sc);
            }
            if (n < ncols) {
                if (of_dy) {
                    *reinterpret_cast<uint2*>(db + ((size_t)i * p.N + n) * c.R + 4 * r4) =
                        make_uint2(pack_h16x2(s.x, s.y, f16), pack_h16x2(s.z, s.w, f16));
                } else {
                    T* o = da + ((size_t)i * c.R + 4 * r4) * p.K + n;
                    o[0] = from_float<T>(s.x);
                    o[p.K] = from_float<T>(s.y);
                    o[2 * p.K] = from_float<T>(s.z);
                    o[3 * p.K] = from_float<T>(s.w);
                }
            }
            row += step_row;
            r4 += step_r4;
            if (of_dy && r4 >= per) {
                r4 -= per;
                ++row;
            }
        }
    }
    if (z > 1)
        cluster_sync();
    if (warp == kLoadWarps)
        tmem_dealloc(tmem, (uint32_t)p.tmem_cols);
}

// ------------------------------------------------------------------------------------ pad

// B with its rows widened to a multiple of 8 ranks by zeros (a tensor map's rows are multiples of 16
// bytes): [rows][4 per] from [rows][R], 8 bytes a thread.
__global__ void __launch_bounds__(256) adapters_pad_kernel(const uint2* __restrict__ b, uint2* __restrict__ out, int64_t rows,
                                                           int r4, int per)
{
    pdl_launch_dependents();
    pdl_wait_prior_grids();
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= rows * per)
        return;
    const int64_t row = e / per;
    const int c = (int)(e - row * per);
    out[e] = c < r4 ? __ldg(b + row * r4 + c) : make_uint2(0u, 0u);
}

// ------------------------------------------------------------------------------------ host

bool a16(std::initializer_list<const void*> ps)
{
    for (const void* q : ps)
        if ((reinterpret_cast<uintptr_t>(q) & 15u) != 0)
            return false;
    return true;
}
int rank_up(int64_t R) { return (int)((R + 15) / 16 * 16); }
size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
uint32_t tmem_columns(int n)
{
    uint32_t c = 32;
    while ((int)c < n)
        c *= 2;
    return c;
}

// The workspace: halves for the wide product, halves of v and u for the grams, and what fp16 needs.
struct Layout {
    size_t halves, back, v, tile_max, pad, total;
    Layout(int64_t M, int64_t N, int64_t L, int64_t R)
    {
        const size_t tiles = (size_t)max_tiles(M, L, kTileL), slots = tiles * kTileL;
        halves = up256(2 * slots * (size_t)rank_up(R) * 2);
        back = up256(slots * sizeof(float));
        v = up256(slots * (size_t)rank_up(R) * sizeof(float));
        tile_max = up256(tiles * kMaxSplit * 2 * sizeof(float));
        pad = R % 8 == 4 ? up256((size_t)L * (size_t)N * (size_t)(R + 4) * 2) : 0;
        total = 3 * halves + back + v + tile_max + pad;
    }
};

Common common_of(const PlanView& plan, qlin_dtype dt, int64_t M, int64_t N, int64_t L, int64_t R, void* ws,
                 const DeviceInfo& dev)
{
    const Layout l(M, N, L, R);
    uint8_t* p = static_cast<uint8_t*>(ws);
    Common c;
    c.plan = plan;
    c.M = M;
    c.slots = max_tiles(M, L, kTileL) * kTileL;
    c.L = (int)L;
    c.R = (int)R;
    c.Rq = rank_up(R);
    c.Rb = (int)((R + 7) / 8 * 8);
    c.b_pad = p + 3 * l.halves + l.back + l.v + l.tile_max;
    c.row_halves = reinterpret_cast<uint16_t*>(p);
    c.v_halves = dt == QLIN_F16 ? reinterpret_cast<uint16_t*>(p + l.halves) : c.row_halves;
    c.u_halves = reinterpret_cast<uint16_t*>(p + 2 * l.halves);
    c.row_back = reinterpret_cast<float*>(p + 3 * l.halves);
    c.v = reinterpret_cast<float*>(p + 3 * l.halves + l.back);
    c.tile_max = reinterpret_cast<float*>(p + 3 * l.halves + l.back + l.v);
    c.status = dev.status;
    return c;
}

// A launch behind the stream's previous kernel (the kernels wait for it before touching memory),
// with clusters of cluster_x CTAs along x (0: none).
template <typename P>
cudaError_t launch(void (*kern)(const P), dim3 grid, int threads, int smem, int cluster_x, const P& prm, cudaStream_t st)
{
    const cudaError_t e = allow_launch(reinterpret_cast<const void*>(kern), smem, cluster_x > 8);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster_x;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster_x > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, prm);
}

template <typename T>
CUtensorMapDataType tm_type() { return Is16<T>::f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16; }

// Token rows [M][cols]: boxes of 64 rows, and single rows, 128 bytes wide.
bool row_maps(RowMaps& m, CUtensorMapDataType dt, int elem, const void* p, int64_t M, int64_t cols)
{
    const uint32_t w = 128 / elem;
    return encode_tmap_2d(&m.box, dt, p, (uint64_t)cols, (uint64_t)M, (uint64_t)cols * elem, w, 64) &&
           encode_tmap_2d(&m.row, dt, p, (uint64_t)cols, (uint64_t)M, (uint64_t)cols * elem, w, 1);
}
// Halves [2 slots][Rq] in boxes of 64 ranks.
template <typename T>
bool half_map(CUtensorMap& m, const Common& c, const uint16_t* p, uint32_t rows)
{
    return encode_tmap_2d(&m, tm_type<T>(), p, (uint64_t)c.Rq, (uint64_t)(2 * c.slots), (uint64_t)c.Rq * 2, 64, rows);
}

// CTAs that share a contraction of K: as many as fit on the GPU in one round, at least four steps
// each.  Three CTAs fit an SM, 54 a GPC, so 8 x 6 clusters of 8; two an SM (with rings of 110 KB) leave
// room for 32, and 34 took a second round: dy [4096][14336] and its x, 137 us against 127.  A CTA's
// boxes of 128-byte rows come at 33 GB/s at most, so few tiles are split over up to 16 CTAs.
int narrow_split(const Common& c, int64_t K)
{
    const int64_t tiles = max_tiles(c.M, c.L, kTileL), steps = (K + 63) / 64;
    int z = 1;
    while (z < kMaxSplit && tiles * 2 * z <= (z < 8 ? 384 : 320) && steps / (2 * z) >= 4)
        z *= 2;
    return z;
}

template <typename T, bool FWD>
cudaError_t launch_narrow(const Common& c, const RowMaps& w, int64_t K, const void* f, const float* scales, const float* u_in,
                          float* u_out, cudaStream_t st, const DeviceInfo& dev)
{
    NarrowParams p;
    p.c = c;
    p.K = K;
    p.scales = scales;
    p.u_in = u_in;
    p.u_out = u_out;
    // a factor of box rows: forward Rq rows of 64 k; backward 64 rows of 64 ranks, an atom each
    p.w = w;
    if (!(FWD ? encode_tmap_3d(&p.tm_f, tm_type<T>(), f, (uint64_t)K, (uint64_t)c.R, (uint64_t)c.L, 2, 64, (uint32_t)c.Rq)
              : encode_tmap_3d(&p.tm_f, tm_type<T>(), f, (uint64_t)c.Rb, (uint64_t)K, (uint64_t)c.L, 2, 64, 64)))
        return cudaErrorInvalidValue;
    p.f_bytes = FWD ? c.Rq * 128 : (c.Rq + 63) / 64 * (int)kAtom;
    const int stage = 2 * (int)kAtom + p.f_bytes;
    const int z = narrow_split(c, K);
    const int room = 74 * 1024;
    p.stages = room / stage < kNarrowMaxStages ? room / stage : kNarrowMaxStages;
    if (p.stages < 3)
        p.stages = 3;
    const int red = 128 * (c.Rq + 4) * 4;
    const int smem = (p.stages * stage > red ? p.stages * stage : red) + 1024;
    p.tmem_cols = (int)tmem_columns(c.Rq);
    p.steps = (int)((K + 63) / 64 + z - 1) / z;
    const dim3 grid((unsigned)z, (unsigned)max_tiles(c.M, c.L, kTileL));
    return launch(adapters_narrow_kernel<T, FWD>, grid, kNarrowThreads, smem, z, p, st);
}

template <typename T, bool FWD>
cudaError_t launch_wide(const Common& c, const void* f, const float* scales, const void* base, void* out, int64_t N,
                        cudaStream_t st, const DeviceInfo& dev)
{
    WideParams p;
    p.c = c;
    p.scales = scales;
    p.base_p = base;
    p.out = out;
    p.N = N;
    if (!row_maps(p.base, tm_type<T>(), 2, base ? base : out, c.M, N) || !half_map<T>(p.tm_h, c, c.row_halves, 128) ||
        !(FWD ? encode_tmap_3d(&p.tm_f, tm_type<T>(), f, (uint64_t)c.Rb, (uint64_t)N, (uint64_t)c.L, 2, 64, kWideCols)
              : encode_tmap_3d(&p.tm_f, tm_type<T>(), f, (uint64_t)N, (uint64_t)c.R, (uint64_t)c.L, 2, 64, (uint32_t)c.Rq)))
        return cudaErrorInvalidValue;
    const int atoms = (c.Rq + 63) / 64, h = 2 * atoms * 2 * (int)kAtom;
    p.f_bytes = FWD ? atoms * 2 * (int)kAtom : 2 * c.Rq * 128;
    const int stage = 4 * (int)kAtom + p.f_bytes, room = 224 * 1024 - h;
    p.stages = room / stage < kWideMaxStages ? room / stage : kWideMaxStages;
    const int64_t tiles = max_tiles(c.M, c.L, kTileL);
    p.blocks = (int)((N + kWideCols - 1) / kWideCols);
    const int64_t units = tiles * p.blocks;
    const dim3 grid((unsigned)(units < dev.sm_count ? units : dev.sm_count));
    return launch(adapters_wide_kernel<T, FWD>, grid, kWideThreads, h + p.stages * stage + 1024, 0, p, st);
}

template <typename T>
cudaError_t launch_grams(const Common& c, const AdapterBwdArgs& a, const RowMaps& dy, cudaStream_t st)
{
    GramParams p;
    p.c = c;
    p.scales = a.scales;
    p.q_scale = a.q ? a.q_scale : nullptr;
    p.g_shift = a.g == 64 ? 6 : a.g == 128 ? 7 : 8;
    p.N = a.N;
    p.K = a.K;
    p.strips_y = (int)((a.N + 255) / 256);
    p.strips_x = (int)((a.K + 255) / 256);
    p.da = a.da;
    p.db = a.db;
    p.parts = narrow_split(c, a.N);
    p.tmem_cols = 256;
    p.dy = dy;
    if (!(a.q ? row_maps(p.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.q, c.M, a.K)
              : row_maps(p.x, tm_type<T>(), 2, a.x, c.M, a.K)) ||
        !half_map<T>(p.tm_u, c, c.u_halves, 64) || !half_map<T>(p.tm_v, c, c.v_halves, 64))
        return cudaErrorInvalidValue;
    p.room = 224 * 1024;
    const int64_t jobs = (int64_t)c.L * (p.strips_y + p.strips_x);
    // split an adapter's tokens over z CTAs, at least two steps each on average, as long as all clusters
    // run at once: with one CTA an SM a GPC of 18 holds 9, 4 or 2 clusters of 2, 4 or 8.  More are slower:
    // 32 jobs (4096 tokens of one adapter, 4096 x 4096) 61 us in all by 4, 82 by 8; 64 jobs 46 by 2, 60 by 4
    int z = 1;
    while (z < kMaxGramSplit && jobs <= (z == 1 ? 72 : z == 2 ? 32 : 16) && c.M / c.L / 64 >= 4 * z)
        z *= 2;
    p.z = z;
    return launch(adapters_gram_kernel<T>, dim3((unsigned)(z * jobs)), kGramThreads, p.room + 1024, z, p, st);
}

// Whether the one-launch kernel is faster than the two tensor-memory ones, by what both cost in us.
// The host does not know how the tokens fall on the adapters: it takes them as drawn evenly, so
// `used` adapters have tokens, and an adapter's last tile is half full on average.  Measured on both
// sides at K, N = 4096 and 11008, ranks 16 - 128, 1 - 1024 tokens, 1 - 100 adapters; e.g. at 4096 x
// 4096, one launch against two: 1 token rank 16 4.2 / 10.2, rank 128 15.8 / 11.9; 61 tokens of 32
// adapters rank 64 14.5 / 24.8; 256 of 4 rank 16 6.2 / 12.1, rank 64 21 / 13.4; 1024 of 4 rank 16 23 / 17.
bool few_tokens(const AdapterFwdArgs& a)
{
    const double M = (double)a.M, n = (double)a.L + 1, used = n * (1 - std::exp(-M / n));
    auto tiles = [&](int t) { return std::max(used, M / t + used / 2); };
    const double row = (double)(a.K + a.N), longer = (double)std::max(a.K, a.N);
    // 18 clusters of 8 at a time, each reading its adapter once
    const double one = 3 + std::ceil(tiles(kTileS) / 18) * 1.4e-5 * rank_up(a.R) * row;
    const double two = 8 + 4e-4 * longer + tiles(kTileL) * row * 5e-5;
    return one < two && max_tiles(a.M, a.L, kTileS) <= 65535;  // a grid's y
}

template <typename T>
cudaError_t launch_decode(const Common& c, const AdapterFwdArgs& a, cudaStream_t st)
{
    DecodeParams p;
    p.c = c;
    p.x = a.x;
    p.a = a.a;
    p.b = a.b;
    p.scales = a.scales;
    p.base = a.base;
    p.out = a.out;
    p.u = a.u;
    p.K = a.K;
    p.N = a.N;
    const int z = 8;
    const dim3 grid((unsigned)z, (unsigned)max_tiles(a.M, a.L, kTileS));
    auto smem = [&](int kt) { return ((kDecodeWarps + z) * 16 * kt * 8 + 8 * (16 * kt + 4)) * (int)sizeof(float); };
    const int kt = c.Rq / 16;
    constexpr int th = kDecodeWarps * 32;
    if (kt <= 1)
        return launch(adapters_decode_kernel<T, 1>, grid, th, smem(1), z, p, st);
    if (kt <= 2)
        return launch(adapters_decode_kernel<T, 2>, grid, th, smem(2), z, p, st);
    if (kt <= 4)
        return launch(adapters_decode_kernel<T, 4>, grid, th, smem(4), z, p, st);
    return launch(adapters_decode_kernel<T, 8>, grid, th, smem(8), z, p, st);
}

// B as the tensor maps can read it: itself, or its padded copy in the workspace.
cudaError_t map_rows(const Common& c, const void* b, int64_t N, cudaStream_t st, const void*& rows)
{
    rows = b;
    if (c.R % 8 == 0)
        return cudaSuccess;
    rows = c.b_pad;
    const int64_t n = (int64_t)c.L * N, per = c.Rb / 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((n * per + 255) / 256));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, adapters_pad_kernel, static_cast<const uint2*>(b), static_cast<uint2*>(c.b_pad), n,
                              c.R / 4, (int)per);
}

template <typename T>
cudaError_t forward_t(const AdapterFwdArgs& a, cudaStream_t st, const DeviceInfo& dev)
{
    const Common c = common_of(a.plan, a.dt, a.M, a.N, a.L, a.R, a.ws, dev);
    if (few_tokens(a))
        return launch_decode<T>(c, a, st);
    const void* b;
    RowMaps x;
    if (!row_maps(x, tm_type<T>(), 2, a.x, a.M, a.K))
        return cudaErrorInvalidValue;
    cudaError_t e = map_rows(c, a.b, a.N, st, b);
    if (e == cudaSuccess)
        e = launch_narrow<T, true>(c, x, a.K, a.a, nullptr, nullptr, a.u, st, dev);
    return e != cudaSuccess ? e : launch_wide<T, true>(c, b, a.scales, a.base, a.out, a.N, st, dev);
}

template <typename T>
cudaError_t backward_t(const AdapterBwdArgs& a, cudaStream_t st, const DeviceInfo& dev)
{
    const Common c = common_of(a.plan, a.dt, a.M, a.N, a.L, a.R, a.ws, dev);
    const void* b;
    RowMaps dy;
    if (!row_maps(dy, tm_type<T>(), 2, a.dy, a.M, a.N))
        return cudaErrorInvalidValue;
    cudaError_t e = map_rows(c, a.b, a.N, st, b);
    if (e == cudaSuccess)
        e = launch_narrow<T, false>(c, dy, a.N, b, a.scales, a.u, nullptr, st, dev);
    if (e == cudaSuccess && Is16<T>::f16) {
        const SplitParams p = {c, a.u, narrow_split(c, a.N)};
        e = launch(adapters_split_kernel, dim3((unsigned)max_tiles(a.M, a.L, kTileL)), 256, 0, 0, p, st);
    }
    if (e == cudaSuccess)
        e = launch_grams<T>(c, a, dy, st);
    if (e == cudaSuccess && a.dx)
        e = launch_wide<T, false>(c, a.a, nullptr, a.dx_base, a.dx, a.K, st, dev);
    return e;
}

static_assert(kMaxPlanTokens / kTileL + kMaxAdapters + 1 <= 65535, "the tile list is a grid's y");
bool tc_sizes(qlin_dtype dt, int64_t N, int64_t K, int64_t R)
{
    return dt != QLIN_F32 && R % 4 == 0 && K % 8 == 0 && N % 8 == 0;
}

}  // namespace

bool adapters_tc_takes(const AdapterFwdArgs& a)
{
    return tc_sizes(a.dt, a.N, a.K, a.R) && a16({a.x, a.a, a.b, a.base, a.out, a.u});
}
bool adapters_tc_takes(const AdapterBwdArgs& a)
{
    return tc_sizes(a.dt, a.N, a.K, a.R) &&
           a16({a.dy, a.a, a.b, a.u, a.x, a.q, a.dx_base, a.dx, a.da, a.db});
}

size_t adapters_tc_workspace(int64_t M, int64_t N, int64_t L, int64_t R) { return Layout(M, N, L, R).total; }

cudaError_t launch_adapters_forward_tc(const AdapterFwdArgs& a, cudaStream_t st, const DeviceInfo& dev)
{
    return a.dt == QLIN_BF16 ? forward_t<__nv_bfloat16>(a, st, dev) : forward_t<__half>(a, st, dev);
}
cudaError_t launch_adapters_backward_tc(const AdapterBwdArgs& a, cudaStream_t st, const DeviceInfo& dev)
{
    return a.dt == QLIN_BF16 ? backward_t<__nv_bfloat16>(a, st, dev) : backward_t<__half>(a, st, dev);
}

}  // namespace qlin
