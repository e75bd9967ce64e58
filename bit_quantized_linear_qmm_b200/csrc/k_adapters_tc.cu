// k_adapters_tc.cu -- low-rank adapters on the tensor cores, bf16 and fp16 (sm_100a).
//
//   narrow   h[m] = A_i x[m]  (forward)  or  v[m] = s_i B_i^T dy[m]  (backward)      tcgen05
//   wide     out[m] = base[m] + s_i B_i h[m]   or   dx[m] = dx_base[m] + A_i^T v[m]  mma.sync
//   grams    dB_i = s_i sum_m dy[m] u[m]^T,  dA_i^T = sum_m x[m] v[m]^T              tcgen05
//
// All three move one long activation row (or write one) for each token and do 2 R products a
// value, R <= 128, so memory bounds them: the tensor cores only have to keep up.  Tokens are taken
// in tiles of 128 of one adapter (the plan's list); a tile's rows lie anywhere in the batch, so
// they are gathered with 16-byte asynchronous copies (zero-filled past the tile's last token, so
// nothing of another adapter's rows enters a sum) instead of tensor-map boxes.
//
// h and v stay in fp32 between the kernels ([tile][128][Rq], Rq = R rounded up to 16, zero where
// there is no token or rank) and enter the second product as two 16-bit halves, hi = round(h) and
// lo = round(h - hi): 2^-16 of the value at most, and two MMAs instead of one.  fp16 halves are
// scaled by a power of two that puts the largest value of the row (wide) or of the adapter (grams)
// in [2^14, 2^15), undone on the fp32 sum; bf16 has fp32's range and needs none.
//
// Every mbarrier wait is bounded: on expiry the kernel records the timeout, every role stops, MMAs
// and copies in flight are waited for and TMEM is freed.
#include <initializer_list>

#include "adapters.cuh"

namespace qlin {
namespace {

constexpr uint32_t kAtom = 64 * 128;  // a 64-row x 128-byte swizzled block
constexpr int kMaxSplit = 8;          // CTAs of a cluster: the portable size

// ------------------------------------------------------------------------------------ helpers

QLIN_DEV void cp_async16(uint32_t dst, const void* src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
QLIN_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
QLIN_DEV void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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
                 : "r"(addr)
                 : "memory");
    return v;
}
QLIN_DEV float ld_peer(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
QLIN_DEV void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b)
{
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
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
    int64_t M;
    int L, R, Rq;
    float* h;         // [tiles of 128][128][Rq]
    float* tile_max;  // [tiles of 128][kMaxSplit][2]: largest finite |v| and |u| of a CTA's rows (fp16)
    unsigned* status;
};

// ------------------------------------------------------------------------------------ narrow

// One cluster for each tile of 128 tokens: its CTAs split the contraction, each accumulating
// [128][Rq] in tensor memory over its steps of 64; the partial sums meet through distributed shared
// memory, CTA j adding the parts of rows 128 j / z .. in order, so h is written once and the order
// of every sum is fixed.
//   warps 0..3   gather the activation rows (cp.async, 128-byte swizzle), then the epilogue
//   warp 4       tensor memory, the MMAs (M = 128, N = Rq, K = 16)
//   warp 5       TMA of the factor: forward A_i [Rq rows][64 k], K-major; backward B_i [64 n][R],
//                MN-major -- a 3-D map, so that rows and columns past the adapter's own are zeros
constexpr int kNarrowLag = 3;       // stages whose copies are in flight behind the newest
constexpr int kNarrowThreads = 192;
constexpr int kNarrowMaxStages = 8;

struct NarrowParams {
    CUtensorMap tm_f;
    Common c;
    const void* w;        // x [M][K] or dy [M][N]
    int64_t K;            // the contraction's length
    int steps;            // 64-wide steps of one CTA
    int stages, f_bytes;  // ring depth, bytes of the factor in a stage
    int tmem_cols;
    const float* scales;  // backward: s
    const float* u_in;    // backward, fp16: u [M][R], for its maximum
    float* u_out;         // forward: [M][R] or null
};

template <typename T, bool FWD>
__global__ void __launch_bounds__(kNarrowThreads) adapters_narrow_tc_kernel(const __grid_constant__ NarrowParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[kNarrowMaxStages], empty[kNarrowMaxStages], acc_full;
    __shared__ uint32_t tmem_s;
    __shared__ int abort_flag;
    __shared__ float warp_max[2][4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int z = gridDim.x, rank = blockIdx.x;  // the cluster spans the grid's x
    const int stage_bytes = 2 * (int)kAtom + p.f_bytes;
    const Common& c = p.c;

    if (tid == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 128 + 1);
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
    if (d.adapter >= c.L) {  // tokens without an adapter: u is zero, nothing reads their h
        if (FWD && p.u_out)
            for (int i = tid; i < rows * c.R; i += kNarrowThreads)
                if (row0 + i / c.R < d.count)
                    p.u_out[(size_t)c.plan.perm[d.start + row0 + i / c.R] * c.R + i % c.R] = 0.f;
        return;
    }
    if (warp == 4)
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

    if (warp < 4) {
        const T* w = static_cast<const T*>(p.w);
        const int chunk = tid & 7;
        int tok[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int row = (tid >> 3) + 16 * j;
            tok[j] = row < d.count ? c.plan.perm[d.start + row] : -1;
        }
        bool ok = true;
        auto publish = [&](int it) {
            fence_proxy_async_smem();
            mbar_arrive(&full[it % p.stages]);
        };
        int it = 0;
        for (; it < n_st; ++it) {
            const int slot = it % p.stages;
            if (it >= p.stages && !mbar_wait_bounded(&empty[slot], ((it / p.stages) & 1) ^ 1, c.status)) {
                ok = false;
                break;
            }
            const int64_t k = (int64_t)(k_first + it) * 64 + chunk * 8;
            const uint32_t dst = smem_u32(X(slot));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = tok[j] >= 0 && k < p.K;
                cp_async16(dst + swz128((tid >> 3) + 16 * j, chunk), in ? w + (size_t)tok[j] * p.K + k : w, in);
            }
            cp_async_commit();
            if (it >= kNarrowLag) {
                cp_async_wait<kNarrowLag>();
                publish(it - kNarrowLag);
            }
        }
        if (ok) {
            if (it >= 3) {
                cp_async_wait<2>();
                publish(it - 3);
            }
            if (it >= 2) {
                cp_async_wait<1>();
                publish(it - 2);
            }
            if (it >= 1) {
                cp_async_wait<0>();
                publish(it - 1);
            }
        } else {
            abort_flag = 1;
            cp_async_wait<0>();
        }
        // this CTA's sums, [128][Rq], into the ring's memory (every copy and MMA is done)
        const bool sums = n_st > 0 && mbar_wait_bounded(&acc_full, 0, c.status) && !aborted(&abort_flag);
        tc_fence_after();
        float* red = reinterpret_cast<float*>(smem) + (size_t)tid * pitch;
        for (int col = 0; col < c.Rq; col += 16) {
            uint32_t r[16];
            if (sums) {
                tmem_ld16(tmem + (uint32_t)col + ((uint32_t)(32 * warp) << 16), r);
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
    } else if (warp == 4) {
        if (lane == 0) {
            const uint32_t ty = Is16<T>::f16 ? 0u : (1u << 7) | (1u << 10);
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
    } else if (lane == 0) {
        int it = 0;
        for (; it < n_st; ++it) {
            const int slot = it % p.stages;
            if ((it >= p.stages && !mbar_wait_bounded(&empty[slot], ((it / p.stages) & 1) ^ 1, c.status)) ||
                aborted(&abort_flag)) {
                abort_flag = 1;
                break;
            }
            mbar_arrive_expect_tx(&full[slot], (unsigned)p.f_bytes);
            const int k = (k_first + it) * 64;
            if constexpr (FWD) {
                tma_load_3d(F(slot), &p.tm_f, k, 0, d.adapter, &full[slot]);
            } else {
                for (int a = 0; a * 64 < c.Rq; ++a)
                    tma_load_3d(F(slot) + a * kAtom, &p.tm_f, a * 64, k, d.adapter, &full[slot]);
            }
        }
        for (int j = it - p.stages < 0 ? 0 : it - p.stages; j < it; ++j)  // no copy may land after the exit
            mbar_wait_bounded(&full[j % p.stages], (j / p.stages) & 1, c.status);
    }
    __syncthreads();
    cluster_sync();
    if (warp < 4) {
        const float sc = FWD ? 1.f : p.scales[d.adapter];
        const int per = c.Rq / 4;
        const uint32_t mine = smem_u32(smem);
        float vmax = 0.f, umax = 0.f;
        for (int i = tid; i < rows * per; i += 128) {
            const int row = row0 + i / per, col = 4 * (i % per);
            const bool in = row < d.count && col < c.R;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int j = 0; j < z; ++j) {
                const float4 v = ld_peer_v4(peer_smem(mine + (uint32_t)(row * pitch + col) * 4u, (uint32_t)j));
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
                s.w += v.w;
            }
            s = in ? make_float4(sc * s.x, sc * s.y, sc * s.z, sc * s.w) : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4*>(c.h + ((size_t)t * kTileL + row) * c.Rq + col) = s;
            if (in && FWD && p.u_out)
                *reinterpret_cast<float4*>(p.u_out + (size_t)c.plan.perm[d.start + row] * c.R + col) = s;
            if (in && !FWD && Is16<T>::f16) {
                const float4 u = *reinterpret_cast<const float4*>(p.u_in + (size_t)c.plan.perm[d.start + row] * c.R + col);
                vmax = fmaxf(fmaxf(vmax, fmaxf(finite_abs(s.x), finite_abs(s.y))), fmaxf(finite_abs(s.z), finite_abs(s.w)));
                umax = fmaxf(fmaxf(umax, fmaxf(finite_abs(u.x), finite_abs(u.y))), fmaxf(finite_abs(u.z), finite_abs(u.w)));
            }
        }
        if (!FWD && Is16<T>::f16) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, o));
                umax = fmaxf(umax, __shfl_xor_sync(0xffffffffu, umax, o));
            }
            if (lane == 0) {
                warp_max[0][warp] = vmax;
                warp_max[1][warp] = umax;
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (tid < 2)
                c.tile_max[((size_t)t * kMaxSplit + rank) * 2 + tid] =
                    fmaxf(fmaxf(warp_max[tid][0], warp_max[tid][1]), fmaxf(warp_max[tid][2], warp_max[tid][3]));
        }
    }
    cluster_sync();  // no CTA's shared memory goes while another reads it
    if (warp == 4)
        tmem_dealloc(tmem, (uint32_t)p.tmem_cols);
}

// ------------------------------------------------------------------------------------ wide

// out = base + h F on mma.sync m16n8k16: 128 rows of a tile by a strip of columns, each warp 16 MT
// rows by 64 columns at a time.  The products (2 R 2 for each value, hi and lo) stay below the rate
// at which memory takes base and out up to R = 64; nothing is staged: the n index of the eight
// 8-column MMAs is permuted so that a thread ends up with 16 consecutive columns of each row (two
// 16-byte loads of base, two stores of out; four lanes cover 128 bytes of a row), and the
// contraction index so that the factor's fragments come straight from memory, 8 bytes of a row of
// B_i (forward) or 16 of rows of A_i (backward).
constexpr int kWideWarps = 8;

struct WideParams {
    Common c;
    const void* f;        // b [L][N][R] (forward) or a [L][R][N] (backward)
    const float* scales;  // forward
    const void* base;
    void* out;
    int64_t N;
    int strip;            // columns of a CTA
};

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

template <typename T, bool FWD, int KT, int MT>
__global__ void __launch_bounds__(kWideWarps * 32) adapters_wide_tc_kernel(const WideParams p)
{
    constexpr int f16 = Is16<T>::f16, kRows = 16 * MT;
    const Common& c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane >> 2, q4 = lane & 3;
    pdl_launch_dependents();
    pdl_wait_prior_grids();
    const int t = blockIdx.y;
    if (t >= c.plan.head[3])
        return;
    const AdapterTile d = c.plan.tiles_l[t];
    const int64_t n_begin = (int64_t)blockIdx.x * p.strip;
    const int64_t n_end = n_begin + p.strip < p.N ? n_begin + p.strip : p.N;
    const T* base = static_cast<const T*>(p.base);
    T* out = static_cast<T*>(p.out);
    if (d.adapter >= c.L) {
        if (base == out)
            return;
        const int vecs = (int)((n_end - n_begin) / 8);
        for (int i = threadIdx.x; i < d.count * vecs; i += kWideWarps * 32) {
            const size_t at = (size_t)c.plan.perm[d.start + i / vecs] * p.N + n_begin + 8 * (i % vecs);
            *reinterpret_cast<uint4*>(out + at) =
                base ? *reinterpret_cast<const uint4*>(base + at) : make_uint4(0u, 0u, 0u, 0u);
        }
        return;
    }
    // the tile's row groups over the warps, the rest of the warps over the columns
    const int groups = (d.count + kRows - 1) / kRows, subs = kWideWarps / groups;
    const int g = warp % groups, sub = warp / groups;
    if (sub >= subs)
        return;
    int tok[MT][2];
    uint32_t hi[MT][KT][4], lo[MT][KT][4];
    float rs[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = g * kRows + m * 16 + j + 8 * e;
            tok[m][e] = row < d.count ? c.plan.perm[d.start + row] : -1;
            const float* h = c.h + ((size_t)t * kTileL + row) * c.Rq;
            float4 v[KT];
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                v[k] = 16 * k < c.Rq ? __ldcg(reinterpret_cast<const float4*>(h + 16 * k + 4 * q4))
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                top = fmaxf(fmaxf(top, fmaxf(finite_abs(v[k].x), finite_abs(v[k].y))),
                            fmaxf(finite_abs(v[k].z), finite_abs(v[k].w)));
            }
            float to = 1.f, back = 1.f;
            if constexpr (f16) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                half_scale<T>(top, to, back);
            }
            rs[m][e] = FWD ? back * p.scales[d.adapter] : back;
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                split2<T>(v[k].x * to, v[k].y * to, hi[m][k][e], lo[m][k][e]);
                split2<T>(v[k].z * to, v[k].w * to, hi[m][k][2 + e], lo[m][k][2 + e]);
            }
        }
    const T* f = static_cast<const T*>(p.f) + (size_t)d.adapter * p.N * c.R;
    for (int64_t nb = n_begin + 64 * sub; nb < n_end; nb += 64 * subs) {
        const int64_t n = nb + 16 * q4;  // this thread's 16 columns
        uint4 bv[MT][2][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int v = 0; v < 2; ++v)
                    bv[m][e][v] = base && tok[m][e] >= 0 && n + 8 * v < p.N
                                      ? *reinterpret_cast<const uint4*>(base + (size_t)tok[m][e] * p.N + n + 8 * v)
                                      : make_uint4(0u, 0u, 0u, 0u);
        float acc[MT][8][4] = {};
        // fragment column j of MMA q is column nb + 8 j + q
        if constexpr (FWD) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int64_t col = nb + 8 * j + q;
                const T* fr = f + (size_t)col * c.R + 4 * q4;
#pragma unroll
                for (int k = 0; k < KT; ++k) {
                    uint2 b = make_uint2(0u, 0u);
                    if (col < p.N && 16 * k + 4 * q4 < c.R)
                        b = __ldg(reinterpret_cast<const uint2*>(fr + 16 * k));
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        mma_16816<T>(acc[m][q], hi[m][k], b.x, b.y);
                        mma_16816<T>(acc[m][q], lo[m][k], b.x, b.y);
                    }
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                uint32_t w[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 16 * k + 4 * q4 + i;
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (r < c.R && nb + 8 * j < p.N)
                        v = __ldg(reinterpret_cast<const uint4*>(f + (size_t)r * p.N + nb + 8 * j));
                    w[i][0] = v.x;
                    w[i][1] = v.y;
                    w[i][2] = v.z;
                    w[i][3] = v.w;
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const uint32_t sel = q & 1 ? 0x7632u : 0x5410u;
                    const uint32_t b0 = prmt(w[0][q >> 1], w[1][q >> 1], sel), b1 = prmt(w[2][q >> 1], w[3][q >> 1], sel);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        mma_16816<T>(acc[m][q], hi[m][k], b0, b1);
                        mma_16816<T>(acc[m][q], lo[m][k], b0, b1);
                    }
                }
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    if (tok[m][e] < 0 || n + 8 * v >= p.N)
                        continue;
                    const uint32_t bw[4] = {bv[m][e][v].x, bv[m][e][v].y, bv[m][e][v].z, bv[m][e][v].w};
                    uint32_t o[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        o[q] = pack_h16x2(fmaf(acc[m][2 * q][2 * e + v], rs[m][e], h16_to_float(bw[q], f16)),
                                          fmaf(acc[m][2 * q + 1][2 * e + v], rs[m][e], h16_to_float(bw[q] >> 16, f16)), f16);
                    *reinterpret_cast<uint4*>(out + (size_t)tok[m][e] * p.N + n + 8 * v) = make_uint4(o[0], o[1], o[2], o[3]);
                }
    }
}

// ------------------------------------------------------------------------------------ grams

// One cluster for each adapter and strip of 256 columns of dy or x: D[256][Rq] = S^T H over the
// adapter's tokens, 64 at a time, the steps dealt round the cluster's CTAs.  S (dy, x or the
// restored x) and H (u or v, hi and lo) lie token by token in shared memory, which is MN-major for
// both operands; nothing is transposed.
//   warps 0..7   gather S (cp.async; codes: 16-byte loads, s q rounded once to the operand type)
//                and H (fp32, split), then the epilogue
//   warp 8       tensor memory, the MMAs (two of M = 128 for hi and for lo, N = Rq, K = 16)
constexpr int kGramProducers = 256;
constexpr int kGramThreads = kGramProducers + 32;
constexpr int kGramStages = 3;

struct GramParams {
    Common c;
    const void* dy;        // [M][N]
    const float* u;        // [M][R]
    const float* scales;
    const void* x;         // [M][K], or
    const int8_t* q;       // [M][K] with
    const float* q_scale;  // [K/g][M]
    int g_shift;
    int64_t N, K;
    int strips_y, strips_x;
    void* da;  // [L][R][K]
    void* db;  // [L][N][R]
    int parts;  // CTAs of a tile in the narrow kernel: maxima of a tile
    int tmem_cols;
};

template <typename T>
__global__ void __launch_bounds__(kGramThreads) adapters_gram_kernel(const GramParams p)
{
    constexpr int f16 = Is16<T>::f16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[kGramStages], empty[kGramStages], acc_full;
    __shared__ uint32_t tmem_s;
    __shared__ int abort_flag;
    __shared__ int toks[3][64];
    const Common& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int z = gridDim.x, rank = blockIdx.x;
    const int atoms_h = (c.Rq + 63) / 64;
    const int h_bytes = atoms_h * (int)kAtom, stage_bytes = 4 * (int)kAtom + 2 * h_bytes;
    if (tid == 0) {
        for (int s = 0; s < kGramStages; ++s) {
            mbar_init(&full[s], kGramProducers);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&acc_full, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8)
        tmem_alloc(&tmem_s, (uint32_t)p.tmem_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_s;
    pdl_launch_dependents();
    pdl_wait_prior_grids();

    const int strips = p.strips_y + p.strips_x;
    const int i = blockIdx.y / strips, strip = blockIdx.y % strips;
    const bool of_dy = strip < p.strips_y, of_q = !of_dy && p.q;
    const int64_t n0 = (int64_t)(of_dy ? strip : strip - p.strips_y) * 256, ncols = of_dy ? p.N : p.K;
    const int seg0 = c.plan.seg[i], tokens = c.plan.seg[i + 1] - seg0;
    const size_t slot0 = (size_t)c.plan.tile_l0[i] * kTileL;
    const int steps = (tokens + 63) / 64;
    const int n_st = steps > rank ? (steps - 1 - rank) / z + 1 : 0;  // steps rank, rank + z, ...
    auto S = [&](int s) { return smem + s * stage_bytes; };
    auto H = [&](int s) { return smem + s * stage_bytes + 4 * kAtom; };
    float to = 1.f, back = 1.f;
    if constexpr (f16) {
        float top = 0.f;
        const int tiles = c.plan.tile_l0[i + 1] - c.plan.tile_l0[i];
        for (int e = lane; e < tiles * p.parts; e += 32)
            top = fmaxf(top, c.tile_max[((size_t)(c.plan.tile_l0[i] + e / p.parts) * kMaxSplit + e % p.parts) * 2 +
                                        (of_dy ? 1 : 0)]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        half_scale<T>(top, to, back);
    }

    if (warp < 8) {
        const T* src = static_cast<const T*>(of_dy ? p.dy : p.x);
        const int per = c.Rq / 4;                        // 16-byte pieces of a row of H
        const int pieces = 64 * per;                     // <= 8 a thread
        auto first_of = [&](int it) { return (rank + it * z) * 64; };
        auto token_at = [&](int it, int row) {
            const int pos = first_of(it) + row;
            return it < n_st && pos < tokens ? c.plan.perm[seg0 + pos] : -1;
        };
        if (tid < 64) {
            toks[0][tid] = token_at(0, tid);
            toks[1][tid] = token_at(1, tid);
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        float4 hv[8];
        uint4 qv[4];
        float qs[4];
        auto load_regs = [&](int it) {  // H and the codes of step it
            const int* tk = toks[it % 3];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int idx = tid + 256 * e;
                hv[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (idx < pieces) {
                    const int row = idx / per, col = 4 * (idx % per), m = tk[row];
                    if (m >= 0 && col < c.R)
                        hv[e] = of_dy ? __ldg(reinterpret_cast<const float4*>(p.u + (size_t)m * c.R + col))
                                      : __ldcg(reinterpret_cast<const float4*>(c.h + (slot0 + first_of(it) + row) * c.Rq + col));
                }
            }
            if (of_q) {
                const int64_t n = n0 + 16 * (tid & 15);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int m = tk[(tid >> 4) + 16 * e];
                    const bool in = m >= 0 && n < ncols;
                    qv[e] = in ? ldg_stream_v4(p.q + (size_t)m * p.K + n) : make_uint4(0u, 0u, 0u, 0u);
                    qs[e] = in ? __ldg(p.q_scale + (n >> p.g_shift) * c.M + m) : 0.f;
                }
            }
        };
        auto publish = [&](int it) {
            fence_proxy_async_smem();
            mbar_arrive(&full[it % kGramStages]);
        };
        if (n_st > 0)
            load_regs(0);
        bool ok = true;
        int it = 0;
        for (; it < n_st; ++it) {
            const int slot = it % kGramStages;
            const int next = tid < 64 ? token_at(it + 2, tid) : 0;
            if (ok && it >= kGramStages)
                ok = mbar_wait_bounded(&empty[slot], ((it / kGramStages) & 1) ^ 1, c.status);
            if (ok) {
                const uint32_t s0 = smem_u32(S(slot)), h0 = smem_u32(H(slot));
                if (!of_q) {
                    const int64_t n = n0 + 8 * lane;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int row = warp + 8 * e, m = toks[it % 3][row];
                        const bool in = m >= 0 && n < ncols;
                        cp_async16(s0 + (lane >> 3) * kAtom + swz128(row, lane & 7), in ? src + (size_t)m * ncols + n : src, in);
                    }
                } else {
                    const int ch = tid & 15, swap = (ch >> 2) & 1;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int row = (tid >> 4) + 16 * e;
                        const uint32_t w[4] = {qv[e].x, qv[e].y, qv[e].z, qv[e].w};
                        uint32_t o[8];
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const uint32_t v = w[b] ^ 0x80808080u;
                            float fv[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y)  // the byte in the mantissa of 2^23: exact
                                fv[y] = (__uint_as_float(prmt(v, 0x4B000000u, 0x7650u + (uint32_t)y)) - 8388736.f) * qs[e];
                            o[2 * b] = pack_h16x2(fv[0], fv[1], f16);
                            o[2 * b + 1] = pack_h16x2(fv[2], fv[3], f16);
                        }
                        const uint32_t at = s0 + (ch >> 2) * kAtom;
                        const int un = 2 * (ch & 3);
                        if (swap) {  // chunks of two atoms in a phase: other units first
                            st_shared_v4(at + swz128(row, un + 1), o[4], o[5], o[6], o[7]);
                            st_shared_v4(at + swz128(row, un), o[0], o[1], o[2], o[3]);
                        } else {
                            st_shared_v4(at + swz128(row, un), o[0], o[1], o[2], o[3]);
                            st_shared_v4(at + swz128(row, un + 1), o[4], o[5], o[6], o[7]);
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int idx = tid + 256 * e;
                    if (idx < pieces) {
                        const int row = idx / per, col = 4 * (idx % per);
                        uint32_t a0, a1, b0, b1;
                        split2<T>(hv[e].x * to, hv[e].y * to, a0, b0);
                        split2<T>(hv[e].z * to, hv[e].w * to, a1, b1);
                        const uint32_t at = h0 + (col >> 6) * kAtom + swz128(row, (col & 63) >> 3) + (col & 7) * 2;
                        st_shared_v2(at, a0, a1);
                        st_shared_v2(at + h_bytes, b0, b1);
                    }
                }
                cp_async_commit();
                if (of_q) {
                    publish(it);
                } else if (it >= 2) {
                    cp_async_wait<2>();
                    publish(it - 2);
                }
            }
            if (it + 1 < n_st)
                load_regs(it + 1);
            if (tid < 64)
                toks[(it + 2) % 3][tid] = next;
            asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        if (ok && !of_q) {
            if (it >= 2) {
                cp_async_wait<1>();
                publish(it - 2);
            }
            if (it >= 1) {
                cp_async_wait<0>();
                publish(it - 1);
            }
        }
        cp_async_wait<0>();
        if (!ok)
            abort_flag = 1;
        const bool sums = n_st > 0 && mbar_wait_bounded(&acc_full, 0, c.status) && !aborted(&abort_flag);
        tc_fence_after();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const int pitch = c.Rq + 4, sub = warp >> 2, row = sub * 128 + 32 * (warp & 3) + lane;
        float* red = reinterpret_cast<float*>(smem) + (size_t)row * pitch;
        for (int col = 0; col < c.Rq; col += 16) {
            uint32_t r[16];
            if (sums) {
                tmem_ld16(tmem + (uint32_t)(sub * c.Rq + col) + ((uint32_t)(32 * (warp & 3)) << 16), r);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    r[e] = 0u;
            }
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<uint4*>(red + col + e) = make_uint4(r[e], r[e + 1], r[e + 2], r[e + 3]);
        }
        tc_fence_before();
    } else {
        if (lane == 0) {
            const uint32_t ty = f16 ? 0u : (1u << 7) | (1u << 10);
            const uint32_t idesc = (1u << 4) | ty | (1u << 15) | (1u << 16) | ((uint32_t)(c.Rq >> 3) << 17) |
                                   ((uint32_t)(128 >> 4) << 24);
            bool ok = true;
            for (int it = 0; it < n_st && ok; ++it) {
                const int slot = it % kGramStages;
                ok = mbar_wait_bounded(&full[slot], (it / kGramStages) & 1, c.status);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t a = smem_u32(S(slot)), b = smem_u32(H(slot));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int sub = 0; sub < 2; ++sub)
#pragma unroll
                        for (int part = 0; part < 2; ++part)
                            tc_mma<false>(tmem + (uint32_t)(sub * c.Rq),
                                          umma_desc_sw128_mn(a + sub * 2 * kAtom + kk * 2048, kAtom),
                                          umma_desc_sw128_mn(b + part * h_bytes + kk * 2048, kAtom), idesc,
                                          (it | kk | part) != 0 ? 1u : 0u);
                tc_commit(&empty[slot]);
            }
            if (!ok)
                abort_flag = 1;
            tc_commit(&acc_full);
            mbar_wait_bounded(&acc_full, 0, c.status);
        }
        __syncwarp();
    }
    __syncthreads();
    cluster_sync();
    if (warp < 8) {
        // CTA j adds the cluster's parts of its share of the 256 columns, in order
        const int share = 256 / z, row0 = rank * share, pitch = c.Rq + 4;
        const uint32_t mine = smem_u32(smem);
        const float sc = of_dy ? (tokens > 0 ? p.scales[i] * back : 0.f) : back;
        T* da = static_cast<T*>(p.da);
        T* db = static_cast<T*>(p.db);
        for (int e = tid; e < share * c.R; e += 256) {
            // consecutive threads write consecutive elements: r of dB's rows, columns of dA's
            const int row = row0 + (of_dy ? e / c.R : e % share), r = of_dy ? e % c.R : e / share;
            if (n0 + row >= ncols)
                continue;
            float s = 0.f;
            for (int k = 0; k < z; ++k)
                s += ld_peer(peer_smem(mine + (uint32_t)(row * pitch + r) * 4u, (uint32_t)k));
            const T v = from_float<T>(tokens > 0 ? s * sc : 0.f);
            if (of_dy)
                db[((size_t)i * p.N + n0 + row) * c.R + r] = v;
            else
                da[((size_t)i * c.R + r) * p.K + n0 + row] = v;
        }
    }
    cluster_sync();
    if (warp == 8)
        tmem_dealloc(tmem, (uint32_t)p.tmem_cols);
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
size_t h_bytes(int64_t M, int64_t L, int64_t R)
{
    return up256((size_t)max_tiles(M, L, kTileL) * kTileL * rank_up(R) * sizeof(float));
}
uint32_t tmem_columns(int n)
{
    uint32_t c = 32;
    while ((int)c < n)
        c *= 2;
    return c;
}

Common common_of(const PlanView& plan, int64_t M, int64_t L, int64_t R, void* ws, const DeviceInfo& dev)
{
    Common c;
    c.plan = plan;
    c.M = M;
    c.L = (int)L;
    c.R = (int)R;
    c.Rq = rank_up(R);
    c.h = static_cast<float*>(ws);
    c.tile_max = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + h_bytes(M, L, R));
    c.status = dev.status;
    return c;
}

// A launch behind the stream's previous kernel (the kernels wait for it before touching memory),
// with clusters of cluster_x CTAs along x.
template <typename P>
cudaError_t launch(void (*kern)(const P), dim3 grid, int threads, int smem, int cluster_x, const P& prm, cudaStream_t st)
{
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess)
            return e;
    }
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

// CTAs that share a contraction of K: more until two an SM have work, at least four steps each.
int narrow_split(const Common& c, int64_t K, const DeviceInfo& dev)
{
    const int64_t tiles = max_tiles(c.M, c.L, kTileL), steps = (K + 63) / 64;
    int z = 1;
    while (z < kMaxSplit && tiles * z < 2 * dev.sm_count && steps / (2 * z) >= 4)
        z *= 2;
    return z;
}

template <typename T, bool FWD>
cudaError_t launch_narrow(const Common& c, const void* w, int64_t K, const void* f, const float* scales, const float* u_in,
                          float* u_out, cudaStream_t st, const DeviceInfo& dev)
{
    NarrowParams p;
    p.c = c;
    p.w = w;
    p.K = K;
    p.scales = scales;
    p.u_in = u_in;
    p.u_out = u_out;
    // a factor of box rows: forward Rq rows of 64 k; backward 64 rows of 64 ranks, an atom each
    if (!(FWD ? encode_tmap_3d(&p.tm_f, tm_type<T>(), f, (uint64_t)K, (uint64_t)c.R, (uint64_t)c.L, 2, 64, (uint32_t)c.Rq)
              : encode_tmap_3d(&p.tm_f, tm_type<T>(), f, (uint64_t)c.R, (uint64_t)K, (uint64_t)c.L, 2, 64, 64)))
        return cudaErrorInvalidValue;
    p.f_bytes = FWD ? c.Rq * 128 : (c.Rq + 63) / 64 * (int)kAtom;
    const int stage = 2 * (int)kAtom + p.f_bytes;
    p.stages = 110 * 1024 / stage < kNarrowMaxStages ? 110 * 1024 / stage : kNarrowMaxStages;
    if (p.stages < 4)
        p.stages = 4;
    const int red = 128 * (c.Rq + 4) * 4;
    const int smem = (p.stages * stage > red ? p.stages * stage : red) + 1024;
    p.tmem_cols = (int)tmem_columns(c.Rq);
    const int64_t tiles = max_tiles(c.M, c.L, kTileL);
    const int z = narrow_split(c, K, dev);
    p.steps = (int)((K + 63) / 64 + z - 1) / z;
    return launch(adapters_narrow_tc_kernel<T, FWD>, dim3((unsigned)z, (unsigned)tiles), kNarrowThreads, smem, z, p, st);
}

template <typename T, bool FWD>
cudaError_t launch_wide(const Common& c, const void* f, const float* scales, const void* base, void* out, int64_t N,
                        cudaStream_t st, const DeviceInfo& dev)
{
    WideParams p;
    p.c = c;
    p.f = f;
    p.scales = scales;
    p.base = base;
    p.out = out;
    p.N = N;
    const int64_t tiles = max_tiles(c.M, c.L, kTileL);
    // strips of 2048 columns, shorter while that leaves fewer than four CTAs an SM
    p.strip = 2048;
    while (p.strip > 128 && tiles * ((N + p.strip - 1) / p.strip) < 4 * dev.sm_count)
        p.strip /= 2;
    const dim3 grid((unsigned)((N + p.strip - 1) / p.strip), (unsigned)tiles);
    const int kt = c.Rq / 16;
    constexpr int th = kWideWarps * 32;
    if (kt <= 1)
        return launch(adapters_wide_tc_kernel<T, FWD, 1, 2>, grid, th, 0, 0, p, st);
    if (kt <= 2)
        return launch(adapters_wide_tc_kernel<T, FWD, 2, 2>, grid, th, 0, 0, p, st);
    if (kt <= 4)
        return launch(adapters_wide_tc_kernel<T, FWD, 4, 2>, grid, th, 0, 0, p, st);
    return launch(adapters_wide_tc_kernel<T, FWD, 8, 1>, grid, th, 0, 0, p, st);
}

template <typename T>
cudaError_t launch_grams(const Common& c, const AdapterBwdArgs& a, cudaStream_t st, const DeviceInfo& dev)
{
    GramParams p;
    p.c = c;
    p.dy = a.dy;
    p.u = a.u;
    p.scales = a.scales;
    p.x = a.x;
    p.q = a.q;
    p.q_scale = a.q_scale;
    p.g_shift = a.g == 64 ? 6 : a.g == 128 ? 7 : 8;
    p.N = a.N;
    p.K = a.K;
    p.strips_y = (int)((a.N + 255) / 256);
    p.strips_x = (int)((a.K + 255) / 256);
    p.da = a.da;
    p.db = a.db;
    p.parts = narrow_split(c, a.N, dev);
    p.tmem_cols = (int)tmem_columns(2 * c.Rq);
    const int ring = kGramStages * (4 * (int)kAtom + 2 * ((c.Rq + 63) / 64) * (int)kAtom), red = 256 * (c.Rq + 4) * 4;
    const int smem = (ring > red ? ring : red) + 1024;
    const int64_t jobs = (int64_t)c.L * (p.strips_y + p.strips_x);
    // split an adapter's tokens until every SM has work, at least two steps each on average
    int z = 1;
    while (z < kMaxSplit && jobs * z < dev.sm_count && c.M / c.L / 64 >= 4 * z)
        z *= 2;
    return launch(adapters_gram_kernel<T>, dim3((unsigned)z, (unsigned)jobs), kGramThreads, smem, z, p, st);
}

template <typename T>
cudaError_t forward_t(const AdapterFwdArgs& a, cudaStream_t st, const DeviceInfo& dev)
{
    const Common c = common_of(a.plan, a.M, a.L, a.R, a.ws, dev);
    const cudaError_t e = launch_narrow<T, true>(c, a.x, a.K, a.a, nullptr, nullptr, a.u, st, dev);
    return e != cudaSuccess ? e : launch_wide<T, true>(c, a.b, a.scales, a.base, a.out, a.N, st, dev);
}

template <typename T>
cudaError_t backward_t(const AdapterBwdArgs& a, cudaStream_t st, const DeviceInfo& dev)
{
    const Common c = common_of(a.plan, a.M, a.L, a.R, a.ws, dev);
    cudaError_t e = launch_narrow<T, false>(c, a.dy, a.N, a.b, a.scales, a.u, nullptr, st, dev);
    if (e == cudaSuccess)
        e = launch_grams<T>(c, a, st, dev);
    if (e == cudaSuccess && a.dx)
        e = launch_wide<T, false>(c, a.a, nullptr, a.dx_base, a.dx, a.K, st, dev);
    return e;
}

bool tc_sizes(qlin_dtype dt, int64_t M, int64_t N, int64_t K, int64_t L, int64_t R)
{
    // the tile list and the gram jobs are a grid's y
    return dt != QLIN_F32 && R % 8 == 0 && K % 8 == 0 && N % 8 == 0 && max_tiles(M, L, kTileL) <= 65535 &&
           L * ((N + 255) / 256 + (K + 255) / 256) <= 65535;
}

}  // namespace

bool adapters_tc_takes(const AdapterFwdArgs& a)
{
    return tc_sizes(a.dt, a.M, a.N, a.K, a.L, a.R) && a16({a.x, a.a, a.b, a.base, a.out, a.u});
}
bool adapters_tc_takes(const AdapterBwdArgs& a)
{
    return tc_sizes(a.dt, a.M, a.N, a.K, a.L, a.R) &&
           a16({a.dy, a.a, a.b, a.u, a.x, a.q, a.dx_base, a.dx, a.da, a.db});
}

size_t adapters_tc_workspace(int64_t M, int64_t L, int64_t R)
{
    return h_bytes(M, L, R) + up256((size_t)max_tiles(M, L, kTileL) * kMaxSplit * 2 * sizeof(float));
}

cudaError_t launch_adapters_forward_tc(const AdapterFwdArgs& a, cudaStream_t st, const DeviceInfo& dev)
{
    return a.dt == QLIN_BF16 ? forward_t<__nv_bfloat16>(a, st, dev) : forward_t<__half>(a, st, dev);
}
cudaError_t launch_adapters_backward_tc(const AdapterBwdArgs& a, cudaStream_t st, const DeviceInfo& dev)
{
    return a.dt == QLIN_BF16 ? backward_t<__nv_bfloat16>(a, st, dev) : backward_t<__half>(a, st, dev);
}

}  // namespace qlin
