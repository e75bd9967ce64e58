// k_checkpoint.cu -- activations kept in 8 bits for the backward pass: restoring them, and the
// weight gradient straight from them.
//
// A checkpoint of x [M tokens][K] is its per-group int8 quantisation (qlin_quantize_int8_groups):
// codes q [M][K] and fp32 scales [K/g][M] with x^[m][k] = q[m][k] scale[k/g][m].
//
//   restore   x^ in the type asked for
//   wgrad     dW[n][k] = sum_m dy[m][n] x^[m][k]      db[n] = sum_m dy[m][n]
#include "qlin_common.cuh"

namespace qlin {

cudaError_t launch_dequantize_int8_groups(const int8_t* q, const float* scale, int64_t N, int64_t K, int g, void* out,
                                          qlin_dtype o_dt, cudaStream_t st);
cudaError_t launch_pergroup_wgrad(const void* dy, qlin_dtype dt, int64_t M, int64_t N, const int8_t* q,
                                  const float* scale, int64_t K, int g, void* dw, void* db, cudaStream_t st,
                                  const DeviceInfo& dev);

namespace {

QLIN_DEV float code_of(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

// Restoring: 1 byte in and 2 or 4 out for each value, bound by memory.  A block takes 8 rows by 512
// columns (a warp a row), whose scales are neighbours in memory; a thread 8 codes at a time, so that
// its 16-byte stores (two for fp32) follow one another through the warp.  16384 x 14336 to bf16: 115 us,
// 6.2 TB/s, 0.95 of the copy rate.
template <typename T>
__global__ void __launch_bounds__(256) dequantize_int8_groups_kernel(const int8_t* __restrict__ q,
                                                                     const float* __restrict__ scale, int64_t N,
                                                                     int64_t K, int g_shift, T* __restrict__ out)
{
    const int lane = threadIdx.x & 31;
    const int64_t col = (int64_t)blockIdx.x * 512 + 8 * lane;
    for (int64_t n = (int64_t)blockIdx.y * 8 + (threadIdx.x >> 5); n < N; n += (int64_t)gridDim.y * 8) {
        uint2 v[2];
        float s[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t c = col + 256 * h;
            if (c < K) {
                v[h] = __ldg(reinterpret_cast<const uint2*>(q + n * K + c));
                s[h] = __ldg(scale + (c >> g_shift) * N + n);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t c = col + 256 * h;
            if (c >= K)
                continue;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = code_of(i < 4 ? v[h].x : v[h].y, i & 3) * s[h];
            T* o = out + n * K + c;
            if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<float4*>(o) = make_float4(f[0], f[1], f[2], f[3]);
                *reinterpret_cast<float4*>(o + 4) = make_float4(f[4], f[5], f[6], f[7]);
            } else {
                constexpr int f16 = !__is_same(T, __nv_bfloat16);
                *reinterpret_cast<uint4*>(o) = make_uint4(pack_h16x2(f[0], f[1], f16), pack_h16x2(f[2], f[3], f16),
                                                          pack_h16x2(f[4], f[5], f16), pack_h16x2(f[6], f[7], f16));
            }
        }
    }
}

// ------------------------------------------------------------------------------------ wgrad
//
// A persistent, warp-specialised tcgen05 GEMM.  The contraction runs over tokens, the slow
// dimension of both operands in memory, so both are read MN-major (a shared-memory row holds one
// token's 64 outputs or inputs, 128 bytes, 128-byte swizzle) and nothing is transposed.  Shared
// memory bounds it: the MMAs' operand reads, the decoded codes and the copies all pass through its
// 128 bytes a clock.  So two CTAs work as a pair on tiles of 512 outputs n by 256 inputs k: each
// holds its own 256 outputs of dy and half of the decoded inputs, which the pair's MMAs (M = 256,
// N = 256) share -- 128 KB of traffic a stage of 64 tokens instead of the 192 KB that one CTA needs
// for a 256 x 256 tile.  Few tokens leave the writing of dW as the bound: then single CTAs take
// tiles of 128 x 256 with two accumulators in turn, and write one while the next is multiplied.
//   warp 0        TMA producer: dy boxes {64 outputs, 64 tokens}, the A operand as it is, and code
//                 boxes {128 bytes, 64 tokens}
//   warp 1        512 columns of tensor memory; one thread (of the pair: in CTA 0) issues the MMAs,
//                 two of them (the pair) on each decoded K = 16 step
//   warps 2..17   decode (of the pair: two groups that take stages in turn): 16 codes (one 16-byte load) -> s q in fp32, rounded once to the operand
//                 type, two 16-byte swizzled stores.  Eight lanes of a load or store phase cover
//                 rows r and r + 4 of one 64-input atom, which meet no bank twice.  In the first
//                 column of tiles they also add up dy's columns: db
//   then          epilogue: 32 rows n each, 32 columns at a time through a staging buffer, so that a
//                 store writes 64 bytes of 8 rows (rows straight from tensor memory, 16 bytes of 32
//                 rows an instruction, took 10,000 cycles a tile)
// Where the last round of tiles fills at most half of the pairs, its tiles are cut into their two
// accumulators' halves, one for a pair.
// Every wait is bounded; on expiry the kernel records the timeout, every role stops, and TMEM is
// freed once the MMAs in flight are done.
// The restored inputs are rounded to the operand's type because the tensor cores multiply two of one
// 16-bit type; holding them in two terms would double the MMAs that bound the long batches.  Of [14336]
// [4096] in bf16 dW is off by 0.0020 of its norm, of which 0.0017 is the result's own rounding (fp16 0.00024
// and 0.00021).
// dW [14336][4096] of 4096 tokens: 406 - 432 us in bursts of five calls, 447 in a loop of 3 s at 1.6 GHz
// under the power cap, 1.18 - 1.08 PFLOP/s (single CTAs on 256 x 256 tiles: 501 and more); [4096][11008]
// of 1000: 100 us.
constexpr int kKT = 256;      // inputs k of a tile
constexpr int kStageM = 64;   // tokens of a stage
constexpr uint32_t kAtomBytes = 128 * kStageM;

template <bool PAIR>
struct WgCfg {
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int SUBS = PAIR ? 2 : 1;     // accumulators of a tile: 128 outputs a CTA each
    static constexpr int BUFS = PAIR ? 1 : 2;     // tiles held in tensor memory
    static constexpr int CN = 128 * SUBS;         // outputs of a CTA
    static constexpr int TN = CN * CTAS;          // outputs of a tile
    static constexpr int CK = kKT / CTAS;         // inputs that a CTA decodes
    static constexpr int GROUPS = PAIR ? 2 : 1;   // of decoding warps, taking stages in turn
    static constexpr int XW = 16;                 // decoding warps
    static constexpr int GW = XW / GROUPS;        // of a group: two chunks a thread
    static constexpr int EW = 4 * SUBS;
    static constexpr int A_BYTES = CN * kStageM * 2;
    static constexpr int RAW_BYTES = CK * kStageM;
    static constexpr int B_BYTES = CK * kStageM * 2;
    static constexpr int SLOT = A_BYTES + RAW_BYTES;
    static constexpr int NB = PAIR ? 3 : 2;
    static constexpr int NS = 4;
    static constexpr int STAGE_OUT = EW * 32 * 64;  // staging of the epilogue's warps
    static constexpr int THREADS = (2 + XW + EW) * 32;
    struct Bars {
        uint64_t full[NS], empty[NS], bfull[NB], bempty[NB], acc_full[2], acc_empty[2], mma_done, sums;
        uint32_t tmem;
        int abort_flag;
        float colsum[CN];       // the odd stages' column sums of dy
    };
    static constexpr int SMEM = NS * SLOT + NB * B_BYTES + STAGE_OUT + (int)sizeof(Bars) + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct WgParams {
    CUtensorMap tm_dy;  // [M][N] 16-bit, box {64, 64}, 128-byte swizzle
    CUtensorMap tm_q;   // [M][K] bytes, box {128, 64}, 128-byte swizzle
    const float* scale; // [K/g][M]
    void* dw;           // [N][K]
    void* db;           // [N] or null
    int64_t M, N, K;
    int g_shift;
    int tiles_n, tiles_k;
    int whole;          // tiles taken whole; later ones in halves
    int f16;
    unsigned* status;
};

QLIN_DEV bool aborted(int* flag) { return *reinterpret_cast<volatile int*>(flag) != 0; }

QLIN_DEV void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
QLIN_DEV uint4 ld_shared_v4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Code i of u (codes ^ 0x80, so 0 .. 255) as an exact fp32: the byte in the mantissa of 2^23.
QLIN_DEV float code_f32(uint32_t u, int i)
{
    return __uint_as_float(prmt(u, 0x4B000000u, 0x7650u + (uint32_t)i)) - 8388736.f;
}

// ---- the pair: CTA 0 of a cluster of two leads
QLIN_DEV void pair_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrives on CTA 0's barrier at this address.  What the arrival announces was written in this CTA's
// own shared memory and shown to the async proxy by the fence before it, so it needs no release at
// cluster scope (which took 1300 cycles for each stage).
QLIN_DEV void arrive_leader(uint64_t* bar)
{
    asm volatile(
        "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [r];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}
template <bool PAIR>
QLIN_DEV void wg_alloc(uint32_t* dst)
{
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(dst)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tmem_alloc(dst, 512);
    }
}
template <bool PAIR>
QLIN_DEV void wg_dealloc(uint32_t base)
{
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(base) : "memory");
    else
        tmem_dealloc(base, 512);
}
template <bool PAIR>
QLIN_DEV void wg_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        tc_mma<false>(d, a, b, idesc, accumulate);
}
// Arrives on bar (of the pair: in both CTAs) once every MMA issued so far is done.
template <bool PAIR>
QLIN_DEV void wg_commit(uint64_t* bar)
{
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
    else
        tc_commit(bar);
}

// One piece of work: a tile, all of its accumulators or one.
struct WgUnit {
    int nt, kt, sub, subs;
};

// Groups of 8 tiles along n walk the k tiles together: their dy columns and the codes stay in L2.
QLIN_DEV void wg_tile(int t, int tiles_n, int tiles_k, int& nt, int& kt)
{
    constexpr int G = 8;
    const int grp = t / (G * tiles_k), first = grp * G, gn = min(G, tiles_n - first), r = t - grp * G * tiles_k;
    nt = first + r % gn;
    kt = r / gn;
}

template <bool PAIR>
QLIN_DEV WgUnit wg_unit(int u, const WgParams& p)
{
    WgUnit w;
    const int cut = u - p.whole;
    w.sub = PAIR && cut >= 0 ? cut & 1 : 0;
    w.subs = PAIR && cut < 0 ? 2 : 1;
    wg_tile(PAIR && cut >= 0 ? p.whole + (cut >> 1) : u, p.tiles_n, p.tiles_k, w.nt, w.kt);
    return w;
}

template <bool PAIR, int F16>
__global__ void __launch_bounds__(WgCfg<PAIR>::THREADS, 1) wgrad_tc_kernel(const __grid_constant__ WgParams p)
{
    using C = WgCfg<PAIR>;
    using Bars = typename C::Bars;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars& bars = *reinterpret_cast<Bars*>(smem + C::NS * C::SLOT + C::NB * C::B_BYTES + C::STAGE_OUT);
    auto A = [&](int s) { return smem + s * C::SLOT; };
    auto RAW = [&](int s) { return smem + s * C::SLOT + C::A_BYTES; };
    auto BT = [&](int b) { return smem + C::NS * C::SLOT + b * C::B_BYTES; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)(blockIdx.x & 1) : 0;
    const int unit0 = (int)blockIdx.x / C::CTAS, units = (int)gridDim.x / C::CTAS;
    const int nm = (int)((p.M + kStageM - 1) / kStageM);
    const int all = p.tiles_n * p.tiles_k, tiles = PAIR ? 2 * all - p.whole : all;
    const int my_tiles = tiles > unit0 ? (tiles - 1 - unit0) / units + 1 : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(&bars.full[s], 1);
            mbar_init(&bars.empty[s], 1);
        }
        for (int b = 0; b < C::NB; ++b) {
            mbar_init(&bars.bfull[b], C::GW * C::CTAS);
            mbar_init(&bars.bempty[b], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars.acc_full[b], 1);
            mbar_init(&bars.acc_empty[b], C::EW * C::CTAS);
        }
        mbar_init(&bars.mma_done, 1);
        mbar_init(&bars.sums, C::GW);
        bars.abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if constexpr (PAIR)
        pair_sync();  // both CTAs' barriers exist, both run
    if (warp == 1)
        wg_alloc<PAIR>(&bars.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;
    pdl_wait_prior_grids();

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int ti = 0; ti < my_tiles && ok; ++ti) {
                const WgUnit w = wg_unit<PAIR>(unit0 + ti * units, p);
                for (int mb = 0; mb < nm; ++mb, ++it) {
                    const int slot = it % C::NS;
                    if ((it >= C::NS &&
                         !mbar_wait_bounded(&bars.empty[slot], ((it / C::NS) & 1) ^ 1, p.status)) ||
                        aborted(&bars.abort_flag)) {
                        bars.abort_flag = 1;
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&bars.full[slot], (unsigned)(C::RAW_BYTES + w.subs * 2 * (int)kAtomBytes));
#pragma unroll
                    for (int h = 0; h < C::CK / 128; ++h)
                        tma_load_2d(RAW(slot) + h * kAtomBytes, &p.tm_q, w.kt * kKT + rank * C::CK + h * 128, mb * kStageM,
                                    &bars.full[slot]);
                    for (int a = 2 * w.sub; a < 2 * (w.sub + w.subs); ++a)
                        tma_load_2d(A(slot) + a * kAtomBytes, &p.tm_dy, w.nt * C::TN + rank * C::CN + a * 64, mb * kStageM,
                                    &bars.full[slot]);
                }
            }
            for (int j = it - C::NS < 0 ? 0 : it - C::NS; j < it; ++j)  // no copy may land after the exit
                mbar_wait_bounded(&bars.full[j % C::NS], (j / C::NS) & 1, p.status);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // D f32; A, B of one 16-bit type (bf16 = 1), both MN-major; N = 256, M = 128 a CTA
            const uint32_t ty = F16 ? 0u : (1u << 7) | (1u << 10);
            const uint32_t idesc = (1u << 4) | ty | (1u << 15) | (1u << 16) | ((uint32_t)(kKT >> 3) << 17) |
                                   ((uint32_t)(128 * C::CTAS >> 4) << 24);
            int it = 0;
            bool ok = true;
            for (int ti = 0; ti < my_tiles && ok; ++ti) {
                const int buf = ti % C::BUFS;
                const WgUnit w = wg_unit<PAIR>(unit0 + ti * units, p);
                ok = mbar_wait_bounded(&bars.acc_empty[buf], ((ti / C::BUFS) & 1) ^ 1, p.status);
                tc_fence_after();
                const uint32_t acc = tmem + (uint32_t)(buf * 256);
                for (int mb = 0; mb < nm && ok; ++mb, ++it) {
                    const int slot = it % C::NS, b = it % C::NB;
                    // every decoding warp (of both CTAs) has seen its stage land before it arrived here
                    ok = mbar_wait_bounded(&bars.full[slot], (it / C::NS) & 1, p.status) &&
                         mbar_wait_bounded(&bars.bfull[b], (it / C::NB) & 1, p.status);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint32_t a0 = smem_u32(A(slot)), b0 = smem_u32(BT(b));
#pragma unroll
                    for (int kk = 0; kk < kStageM / 16; ++kk) {
                        const uint64_t bd = umma_desc_sw128_mn(b0 + kk * 2048, kAtomBytes);
#pragma unroll
                        for (int m = 0; m < C::SUBS; ++m) {
                            if (m < w.sub || m >= w.sub + w.subs)
                                continue;
                            wg_mma<PAIR>(acc + (uint32_t)(m * 256),
                                         umma_desc_sw128_mn(a0 + m * 2 * kAtomBytes + kk * 2048, kAtomBytes), bd, idesc,
                                         (mb | kk) != 0 ? 1u : 0u);
                        }
                    }
                    wg_commit<PAIR>(&bars.empty[slot]);
                    wg_commit<PAIR>(&bars.bempty[b]);
                }
                wg_commit<PAIR>(&bars.acc_full[buf]);
            }
            if (!ok)
                bars.abort_flag = 1;
            wg_commit<PAIR>(&bars.mma_done);  // every MMA issued has completed before TMEM is released
            mbar_wait_bounded(&bars.mma_done, 0, p.status);
        }
        __syncwarp();
    } else if (warp < 2 + C::XW) {
        constexpr int ATOMS = C::CK / 64, RW = C::GW / ATOMS, RPW = kStageM / RW;  // rows a warp: 16
        static_assert(RPW == 16, "two chunks a thread");
        const int group = (warp - 2) / C::GW, w = (warp - 2) % C::GW, atom = w % ATOMS;
        const int row0 = (w / ATOMS) * RPW + (lane >> 3) + ((lane >> 2) & 1) * 4;  // + 8 j, j = 0, 1
        const int unit = (atom & 1) * 4 + (lane & 3), bunit = 2 * (lane & 3), swap = (lane >> 2) & 1;
        const int ct = w * 32 + lane;  // column sums: a column a thread
        int it0 = 0, n_sums = 0;       // stages before this tile
        bool ok = true;
        for (int ti = 0; ti < my_tiles && ok; ++ti) {
            const WgUnit wu = wg_unit<PAIR>(unit0 + ti * units, p);
            const int kt = wu.kt;
            const bool sums = kt == 0 && p.db != nullptr;
            const bool here = ct >= 128 * wu.sub && ct < 128 * (wu.sub + wu.subs);  // this thread's column is loaded
            float sum = 0.f;
            const int64_t k = (int64_t)kt * kKT + rank * C::CK + atom * 64;
            const float* sc = k < p.K ? p.scale + (k >> p.g_shift) * p.M : nullptr;
            float s[2], next[2];
            auto load_scales = [&](int mb, float (&d)[2]) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int64_t m = (int64_t)mb * kStageM + row0 + 8 * j;
                    d[j] = sc && m < p.M ? __ldg(sc + m) : 0.f;
                }
            };
            const int mine = C::GROUPS == 2 ? (it0 ^ group) & 1 : 0;  // this group's first stage of the tile
            load_scales(mine, next);
            for (int mb = mine; mb < nm; mb += C::GROUPS) {
                const int it = it0 + mb;
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    s[j] = next[j];
                if (mb + C::GROUPS < nm)
                    load_scales(mb + C::GROUPS, next);
                const int slot = it % C::NS, b = it % C::NB;
                if (!mbar_wait_bounded(&bars.full[slot], (it / C::NS) & 1, p.status) ||
                    !mbar_wait_bounded(&bars.bempty[b], ((it / C::NB) & 1) ^ 1, p.status) ||
                    aborted(&bars.abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t raw = smem_u32(RAW(slot)) + (atom >> 1) * kAtomBytes;
                const uint32_t dst = smem_u32(BT(b)) + atom * kAtomBytes;
                uint4 v[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    v[j] = ld_shared_v4(raw + swz128(row0 + 8 * j, unit));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int row = row0 + 8 * j;
                    const uint32_t c[4] = {v[j].x ^ 0x80808080u, v[j].y ^ 0x80808080u, v[j].z ^ 0x80808080u,
                                           v[j].w ^ 0x80808080u};
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        h[2 * e] = pack_h16x2(code_f32(c[e], 0) * s[j], code_f32(c[e], 1) * s[j], F16);
                        h[2 * e + 1] = pack_h16x2(code_f32(c[e], 2) * s[j], code_f32(c[e], 3) * s[j], F16);
                    }
                    // rows r + 4 of a phase store their second half first
                    const uint32_t lo = dst + swz128(row, bunit), hi = dst + swz128(row, bunit + 1);
                    if (swap) {
                        st_shared_v4(hi, h[4], h[5], h[6], h[7]);
                        st_shared_v4(lo, h[0], h[1], h[2], h[3]);
                    } else {
                        st_shared_v4(lo, h[0], h[1], h[2], h[3]);
                        st_shared_v4(hi, h[4], h[5], h[6], h[7]);
                    }
                }
                if (sums && here) {  // before the arrival below frees the stage
                    const uint8_t* a = A(slot) + (ct >> 6) * kAtomBytes + (ct & 7) * 2;
                    float part = 0.f;
#pragma unroll 16
                    for (int row = 0; row < kStageM; ++row)
                        part += h16_to_float(*reinterpret_cast<const unsigned short*>(a + swz128(row, (ct & 63) >> 3)), F16);
                    sum += part;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR)
                        arrive_leader(&bars.bfull[b]);
                    else
                        mbar_arrive(&bars.bfull[b]);
                }
            }
            it0 += nm;
            if (sums && ok) {
                // the second group hands its sums to the first, which has stages of the next tile to
                // decode before the second can be here again
                if (C::GROUPS == 2 && group == 1) {
                    if (ct < C::CN)
                        bars.colsum[ct] = sum;
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&bars.sums);
                } else {
                    if (C::GROUPS == 2) {
                        ok = mbar_wait_bounded(&bars.sums, n_sums & 1, p.status);
                        ++n_sums;
                        sum += ct < C::CN ? bars.colsum[ct] : 0.f;
                    }
                    const int64_t n = (int64_t)wu.nt * C::TN + rank * C::CN + ct;
                    if (here && ok && n < p.N)
                        static_cast<unsigned short*>(p.db)[n] = to_h16(sum, F16);
                }
            }
        }
        if (!ok)
            bars.abort_flag = 1;
    } else {
        const int q = warp & 3, sub = (warp - 2 - C::XW) >> 2;
        const uint32_t out = smem_u32(smem + C::NS * C::SLOT + C::NB * C::B_BYTES) + (uint32_t)(warp - 2 - C::XW) * 2048u;
        for (int ti = 0; ti < my_tiles; ++ti) {
            const int buf = ti % C::BUFS;
            if (!mbar_wait_bounded(&bars.acc_full[buf], (ti / C::BUFS) & 1, p.status) || aborted(&bars.abort_flag)) {
                bars.abort_flag = 1;
                break;
            }
            tc_fence_after();
            const WgUnit w = wg_unit<PAIR>(unit0 + ti * units, p);
            const uint32_t acc = tmem + (uint32_t)((buf + sub) * 256) + ((uint32_t)(32 * q) << 16);
            const int64_t n_first = (int64_t)w.nt * C::TN + rank * C::CN + sub * 128 + 32 * q;
            const int64_t k_first = (int64_t)w.kt * kKT;
            const int cols = (int)(p.K - k_first < kKT ? p.K - k_first : kKT);  // K % 64 == 0
            unsigned short* dw = static_cast<unsigned short*>(p.dw);
            const bool mine = sub >= w.sub && sub < w.sub + w.subs;
#pragma unroll 1
            for (int c = 0; c < cols && mine; c += 32) {
                uint32_t r[2][16];
                tmem_ld16_nowait(acc + (uint32_t)c, r[0]);
                tmem_ld16_nowait(acc + (uint32_t)c + 16u, r[1]);
                tmem_wait_ld();
                __syncwarp();  // the last 32 columns have been read
                // staged rows of 64 bytes, 16-byte units permuted by row / 2: eight rows of a store or
                // load phase meet no bank twice
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[e] = pack_h16x2(__uint_as_float(r[h >> 1][(h & 1) * 8 + 2 * e]),
                                          __uint_as_float(r[h >> 1][(h & 1) * 8 + 2 * e + 1]), F16);
                    st_shared_v4(out + lane * 64 + ((h ^ (lane >> 1) & 3) << 4), o[0], o[1], o[2], o[3]);
                }
                __syncwarp();
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int row = 8 * h + (lane >> 2);
                    const uint4 v = ld_shared_v4(out + row * 64 + (((lane & 3) ^ (row >> 1) & 3) << 4));
                    if (n_first + row < p.N)
                        *reinterpret_cast<uint4*>(dw + (n_first + row) * p.K + k_first + c + 8 * (lane & 3)) = v;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR)
                    arrive_leader(&bars.acc_empty[buf]);
                else
                    mbar_arrive(&bars.acc_empty[buf]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR)
        pair_sync();  // the pair's MMAs read both CTAs' shared memory; arrivals reach CTA 0's
    if (warp == 1)
        wg_dealloc<PAIR>(tmem);
}

int log2_of(int g) { return g == 64 ? 6 : g == 128 ? 7 : 8; }

template <bool PAIR>
cudaError_t launch_wgrad(WgParams& p, cudaStream_t st, const DeviceInfo& dev)
{
    using C = WgCfg<PAIR>;
    auto kern = p.f16 ? wgrad_tc_kernel<PAIR, 1> : wgrad_tc_kernel<PAIR, 0>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess)
        return e;
    p.tiles_n = (int)((p.N + C::TN - 1) / C::TN);
    p.tiles_k = (int)((p.K + kKT - 1) / kKT);
    const int64_t most = dev.sm_count / C::CTAS;
    int64_t tiles = (int64_t)p.tiles_n * p.tiles_k;
    const int64_t rest = tiles % most;
    p.whole = (int)(PAIR && 2 * rest <= most ? tiles - rest : tiles);
    tiles += tiles - p.whole;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(C::CTAS * (tiles < most ? tiles : most)));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C::CTAS;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_dequantize_int8_groups(const int8_t* q, const float* scale, int64_t N, int64_t K, int g, void* out,
                                          qlin_dtype o_dt, cudaStream_t st)
{
    const dim3 blocks((unsigned)((K + 511) / 512), (unsigned)((N + 7) / 8 < 65535 ? (N + 7) / 8 : 65535));
    const int sh = log2_of(g);
    if (o_dt == QLIN_F32)
        dequantize_int8_groups_kernel<float><<<blocks, 256, 0, st>>>(q, scale, N, K, sh, static_cast<float*>(out));
    else if (o_dt == QLIN_BF16)
        dequantize_int8_groups_kernel<__nv_bfloat16>
            <<<blocks, 256, 0, st>>>(q, scale, N, K, sh, static_cast<__nv_bfloat16*>(out));
    else
        dequantize_int8_groups_kernel<__half><<<blocks, 256, 0, st>>>(q, scale, N, K, sh, static_cast<__half*>(out));
    return cudaGetLastError();
}

cudaError_t launch_pergroup_wgrad(const void* dy, qlin_dtype dt, int64_t M, int64_t N, const int8_t* q,
                                  const float* scale, int64_t K, int g, void* dw, void* db, cudaStream_t st,
                                  const DeviceInfo& dev)
{
    WgParams p;
    p.scale = scale;
    p.dw = dw;
    p.db = db;
    p.M = M;
    p.N = N;
    p.K = K;
    p.g_shift = log2_of(g);
    p.f16 = dt == QLIN_F16;
    p.status = dev.status;
    if (!encode_tmap_2d(&p.tm_dy, p.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dy,
                        (uint64_t)N, (uint64_t)M, (uint64_t)N * 2, 64, kStageM) ||
        !encode_tmap_2d(&p.tm_q, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, (uint64_t)K, (uint64_t)M, (uint64_t)K, 128,
                        kStageM))
        return cudaErrorInvalidValue;
    return M > 512 && N > 256 ? launch_wgrad<true>(p, st, dev) : launch_wgrad<false>(p, st, dev);
}

}  // namespace qlin
