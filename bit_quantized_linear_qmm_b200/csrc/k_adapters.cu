// k_adapters.cu -- low-rank adapters of many requests beside a shared projection: the plan (tokens
// ordered by adapter) and the kernels for any type, size and alignment.
//
//   forward    u[m] = A_i x[m]            out[m] = base[m] + s_i B_i u[m]      i = adapter of token m
//   backward   v[m] = s_i B_i^T dy[m]     dx[m] = dx_base[m] + A_i^T v[m]
//              dA_i = sum_m v[m] x[m]^T   dB_i = s_i sum_m dy[m] u[m]^T        over the tokens of i
//
// The general kernels are six instances of one 64 x 64 fp32 tile product (4 x 4 outputs a thread,
// operands staged in shared memory; 64 x 32 or 64 x 16 where the second side is a lower rank).  They serve fp32, whose products the 16-bit tensor cores do
// not hold, row lengths that are not multiples of 8 elements, odd ranks.  Sums run in fp32, in
// a fixed order: partial sums of 128 terms are added to a second accumulator, so that the rounding
// error grows with the number of partial sums and not of terms.
#include "adapters.cuh"
#include "simt_tile.cuh"

namespace qlin {
namespace {

// ------------------------------------------------------------------------------------ plan

// One CTA of 32 warps; warp w counts, then places, the tokens of the w-th part of the batch in
// order, so tokens of one adapter stay ascending (and sums over them have a fixed order).  Lanes
// with the same adapter are grouped by match_any; no atomics.  One CTA, since batches are short and the
// plan is made once for all layers: 61 tokens of 32 adapters 4.1 us, 4096 of 4 5.2 us, 4096 of 1024 17.7 us,
// 65536 of 64 129 us, 2^20 of 1024 2.5 ms.
__global__ void __launch_bounds__(1024) adapters_plan_kernel(const int32_t* __restrict__ ids, int M, int L, PlanView v)
{
    extern __shared__ int cnt[];  // [32][L + 1]
    __shared__ int seg[kMaxAdapters + 2], t_s[kMaxAdapters + 2], t_l[kMaxAdapters + 2];
    const int S = L + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < 32 * S; i += 1024)
        cnt[i] = 0;
    __syncthreads();
    const int part = ((M + 31) / 32 + 31) & ~31;
    const int m0 = min(M, warp * part), m1 = min(M, m0 + part);
    int* mine = cnt + warp * S;
    auto key_of = [&](int m) {
        if (m >= m1)
            return -1;
        const int id = ids[m];
        return id >= 0 && id < L ? id : L;
    };
    for (int m = m0; m < m1; m += 32) {
        const int key = key_of(m + lane);
        const unsigned same = __match_any_sync(0xffffffffu, key);
        if (key >= 0 && lane == __ffs(same) - 1)
            mine[key] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int l = threadIdx.x; l < S; l += 1024) {  // counts -> exclusive sums over the warps; totals
        int sum = 0;
        for (int w = 0; w < 32; ++w) {
            const int c = cnt[w * S + l];
            cnt[w * S + l] = sum;
            sum += c;
        }
        seg[l] = sum;
        t_s[l] = (sum + kTileS - 1) / kTileS;
        t_l[l] = (sum + kTileL - 1) / kTileL;
    }
    __syncthreads();
    if (warp < 3) {  // exclusive sums over the segments, one warp for each array
        int* arr = warp == 0 ? seg : warp == 1 ? t_s : t_l;
        int carry = 0;
        for (int l0 = 0; l0 < S; l0 += 32) {
            const int c = l0 + lane < S ? arr[l0 + lane] : 0;
            int x = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o)
                    x += y;
            }
            if (l0 + lane < S)
                arr[l0 + lane] = carry + x - c;
            carry += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0)
            arr[S] = carry;
    }
    __syncthreads();
    for (int m = m0; m < m1; m += 32) {
        const int key = key_of(m + lane);
        const unsigned same = __match_any_sync(0xffffffffu, key);
        const int rank = __popc(same & ((1u << lane) - 1u));
        if (key >= 0)
            v.perm[seg[key] + mine[key] + rank] = m + lane;
        __syncwarp();
        if (key >= 0 && rank == 0)
            mine[key] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    auto tiles = [&](const int* first, int T, AdapterTile* out) {
        for (int t = threadIdx.x; t < first[S]; t += 1024) {
            int lo = 0, hi = S;  // the last segment whose first tile is <= t and that has tiles
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first[mid] <= t)
                    lo = mid;
                else
                    hi = mid;
            }
            AdapterTile d;
            d.adapter = lo;
            d.start = seg[lo] + (t - first[lo]) * T;
            d.count = min(T, seg[lo + 1] - d.start);
            const int a = v.perm[d.start], b = v.perm[d.start + d.count - 1];
            d.first = b - a == d.count - 1 ? a : -1;
            out[t] = d;
        }
    };
    tiles(t_s, kTileS, v.tiles_s);
    tiles(t_l, kTileL, v.tiles_l);
    for (int l = threadIdx.x; l <= S; l += 1024) {
        v.seg[l] = seg[l];
        v.tile_l0[l] = t_l[l];
    }
    if (threadIdx.x == 0) {
        v.head[0] = M;
        v.head[1] = L;
        v.head[2] = t_s[S];
        v.head[3] = t_l[S];
        v.head[4] = t_s[L];
        v.head[5] = t_l[L];
    }
}

// ------------------------------------------------------------------------------------ general kernels

// Token sub-tile blockIdx.x: the first or second 64 tokens of a 128-tile.
struct SubTile {
    int adapter, start, count;
};
QLIN_DEV bool sub_tile(const PlanView& v, bool with_none, SubTile& s)
{
    const int t = blockIdx.x >> 1, half = (blockIdx.x & 1) * kB;
    if (t >= v.head[with_none ? 3 : 5])
        return false;
    const AdapterTile d = v.tiles_l[t];
    if (half >= d.count)
        return false;
    s.adapter = d.adapter;
    s.start = d.start + half;
    s.count = min(kB, d.count - half);
    return true;
}

// part[z][position][r] = the z-th part of sum_k w[token][k] f_i[r][k]; w = x, f = A (forward: the
// factor's rows run along k) or w = dy, f = B^T (backward: along r).
template <typename T, bool FWD, int C>
__global__ void __launch_bounds__(kThreads) adapters_narrow_kernel(const T* __restrict__ w, const T* __restrict__ f,
                                                                   int64_t M, int64_t K, int R, PlanView v,
                                                                   float* __restrict__ part)
{
    SubTile s;
    if (!sub_tile(v, false, s))
        return;
    const int r0 = blockIdx.y * (16 * C);
    const int64_t per = ((K + gridDim.z - 1) / gridDim.z + kBK - 1) / kBK * kBK;
    const int64_t k0 = per * blockIdx.z, k1 = k0 + per < K ? k0 + per : K;
    const T* fi = f + (size_t)s.adapter * R * K;
    const int* perm = v.perm + s.start;
    float o[4][C];
    tile_product<C, true, FWD>(
        k0, k1, [&](int i, int64_t k) { return i < s.count ? to_float(w[(size_t)perm[i] * K + k]) : 0.f; },
        [&](int j, int64_t k) {
            return r0 + j < R ? to_float(FWD ? fi[(size_t)(r0 + j) * K + k] : fi[(size_t)k * R + r0 + j]) : 0.f;
        },
        o);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (4 * ty + r < s.count && r0 + C * tx + c < R)
                part[((size_t)blockIdx.z * M + s.start + 4 * ty + r) * R + r0 + C * tx + c] = o[r][c];
}

// sum[position][r] = sum over the parts, in order; u (forward, [token][r]) gets the same, and zero
// for the tokens without an adapter.
__global__ void __launch_bounds__(256) adapters_sum_kernel(const float* __restrict__ part, int parts, int64_t M, int L,
                                                           int R, PlanView v, float* __restrict__ sum,
                                                           float* __restrict__ u)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= M * R)
        return;
    const int64_t pos = i / R;
    const bool has = pos < v.seg[L];
    float t = 0.f;
    if (has)
        for (int z = 0; z < parts; ++z)
            t += part[(size_t)z * M * R + i];
    sum[i] = t;
    if (u)
        u[(size_t)v.perm[pos] * R + i % R] = t;
}

// out[token][n] = base[token][n] + scale_i sum_r h[position][r] f_i(r, n): f = B (forward: rows run
// along r, scale_i = s_i) or f = A (backward: along n, no scale: v holds it).
template <typename T, bool FWD>
__global__ void __launch_bounds__(kThreads) adapters_wide_kernel(const float* __restrict__ h, const T* __restrict__ f,
                                                                 const float* __restrict__ scales, const T* base,
                                                                 T* out, int64_t N, int L, int R, PlanView v)
{
    SubTile s;
    if (!sub_tile(v, true, s))
        return;
    const int64_t n0 = (int64_t)blockIdx.y * kB;
    const bool has = s.adapter < L;
    if (!has && base == out)
        return;
    float o[4][4] = {};
    if (has) {
        const T* fi = f + (size_t)s.adapter * R * N;
        const float sc = FWD ? scales[s.adapter] : 1.f;
        tile_product<4, true, FWD>(
            0, R, [&](int i, int64_t r) { return i < s.count ? sc * h[(size_t)(s.start + i) * R + r] : 0.f; },
            [&](int j, int64_t r) {
                return n0 + j < N ? to_float(FWD ? fi[(size_t)(n0 + j) * R + r] : fi[(size_t)r * N + n0 + j]) : 0.f;
            },
            o);
    }
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (4 * ty + r >= s.count)
            continue;
        const size_t row = (size_t)v.perm[s.start + 4 * ty + r] * N;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int64_t n = n0 + 4 * tx + c;
            if (n < N)
                out[row + n] = from_float<T>((base ? to_float(base[row + n]) : 0.f) + o[r][c]);
        }
    }
}

// The layer's input as it is, or restored from its int8 checkpoint.
template <typename T>
struct Input {
    const T* x;
    const int8_t* q;
    const float* q_scale;
    int g;
    int64_t M, K;
    QLIN_DEV float operator()(int m, int64_t k) const
    {
        return x ? to_float(x[(size_t)m * K + k]) : (float)q[(size_t)m * K + k] * q_scale[(size_t)(k / g) * M + m];
    }
};

// dA_i[r][k] = sum over the tokens of i of v[position][r] x[token][k]; zero without tokens.
template <typename T, int C>
__global__ void __launch_bounds__(kThreads) adapters_da_kernel(const float* __restrict__ h, Input<T> x,
                                                               T* __restrict__ da, int64_t K, int R, PlanView v)
{
    const int i = blockIdx.z, r0 = blockIdx.y * (16 * C);
    const int64_t c0 = (int64_t)blockIdx.x * kB;
    float o[4][C];
    tile_product<C, false, false>(
        v.seg[i], v.seg[i + 1], [&](int k, int64_t p) { return c0 + k < K ? x(v.perm[p], c0 + k) : 0.f; },
        [&](int r, int64_t p) { return r0 + r < R ? h[(size_t)p * R + r0 + r] : 0.f; }, o);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (r0 + C * tx + c < R && c0 + 4 * ty + r < K)
                da[((size_t)i * R + r0 + C * tx + c) * K + c0 + 4 * ty + r] = from_float<T>(o[r][c]);
}

// dB_i[n][r] = s_i sum over the tokens of i of dy[token][n] u[token][r]; zero without tokens.
template <typename T, int C>
__global__ void __launch_bounds__(kThreads) adapters_db_kernel(const T* __restrict__ dy, const float* __restrict__ u,
                                                               const float* __restrict__ scales, T* __restrict__ db,
                                                               int64_t N, int R, PlanView v)
{
    const int i = blockIdx.z, r0 = blockIdx.y * (16 * C);
    const int64_t n0 = (int64_t)blockIdx.x * kB;
    float o[4][C];
    tile_product<C, false, false>(
        v.seg[i], v.seg[i + 1],
        [&](int n, int64_t p) { return n0 + n < N ? to_float(dy[(size_t)v.perm[p] * N + n0 + n]) : 0.f; },
        [&](int r, int64_t p) { return r0 + r < R ? u[(size_t)v.perm[p] * R + r0 + r] : 0.f; }, o);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const float sc = scales[i];
    const bool any = v.seg[i] < v.seg[i + 1];  // a scale that is not finite times no token is no gradient
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (n0 + 4 * ty + r < N && r0 + C * tx + c < R)
                db[((size_t)i * N + n0 + 4 * ty + r) * R + r0 + C * tx + c] = from_float<T>(any ? sc * o[r][c] : 0.f);
}

// v = s_i h in place: the backward pass's narrow sum holds the scale.
__global__ void __launch_bounds__(256) adapters_scale_kernel(float* __restrict__ h, const float* __restrict__ scales,
                                                             int L, int R, PlanView v)
{
    const AdapterTile d = v.tiles_l[blockIdx.x < (unsigned)v.head[5] ? blockIdx.x : 0];
    if (blockIdx.x >= (unsigned)v.head[5])
        return;
    const float sc = scales[d.adapter];
    for (int i = threadIdx.x; i < d.count * R; i += 256)
        h[(size_t)d.start * R + i] *= sc;
}

// Parts of a contraction over K: about 512 terms each, 16 at most.
int parts_of(int64_t K) { return (int)(K / 512 < 1 ? 1 : K / 512 > 16 ? 16 : K / 512); }
unsigned blocks_of(int64_t n, int64_t per) { return (unsigned)((n + per - 1) / per); }

// C: ranks of a tile's side by 16
template <typename T, int C>
cudaError_t forward_c(const AdapterFwdArgs& a, cudaStream_t st)
{
    const int R = (int)a.R, L = (int)a.L, parts = parts_of(a.K);
    const unsigned subs = 2u * (unsigned)max_tiles(a.M, a.L, kTileL), ry = blocks_of(R, 16 * C);
    float* part = static_cast<float*>(a.ws);
    float* sum = part + (size_t)parts * a.M * R;
    adapters_narrow_kernel<T, true, C><<<dim3(subs, ry, parts), kThreads, 0, st>>>(
        static_cast<const T*>(a.x), static_cast<const T*>(a.a), a.M, a.K, R, a.plan, part);
    adapters_sum_kernel<<<blocks_of(a.M * R, 256), 256, 0, st>>>(part, parts, a.M, L, R, a.plan, sum, a.u);
    adapters_wide_kernel<T, true><<<dim3(subs, blocks_of(a.N, kB)), kThreads, 0, st>>>(
        sum, static_cast<const T*>(a.b), a.scales, static_cast<const T*>(a.base), static_cast<T*>(a.out), a.N, L, R,
        a.plan);
    return cudaGetLastError();
}

template <typename T, int C>
cudaError_t backward_c(const AdapterBwdArgs& a, cudaStream_t st)
{
    const int R = (int)a.R, L = (int)a.L, parts = parts_of(a.N);
    const unsigned subs = 2u * (unsigned)max_tiles(a.M, a.L, kTileL), ry = blocks_of(R, 16 * C);
    float* part = static_cast<float*>(a.ws);
    float* sum = part + (size_t)parts * a.M * R;
    adapters_narrow_kernel<T, false, C><<<dim3(subs, ry, parts), kThreads, 0, st>>>(
        static_cast<const T*>(a.dy), static_cast<const T*>(a.b), a.M, a.N, R, a.plan, part);
    adapters_sum_kernel<<<blocks_of(a.M * R, 256), 256, 0, st>>>(part, parts, a.M, L, R, a.plan, sum, nullptr);
    adapters_scale_kernel<<<(unsigned)max_tiles(a.M, a.L, kTileL), 256, 0, st>>>(sum, a.scales, L, R, a.plan);
    if (a.dx)
        adapters_wide_kernel<T, false><<<dim3(subs, blocks_of(a.K, kB)), kThreads, 0, st>>>(
            sum, static_cast<const T*>(a.a), nullptr, static_cast<const T*>(a.dx_base), static_cast<T*>(a.dx), a.K, L,
            R, a.plan);
    const Input<T> in = {static_cast<const T*>(a.x), a.q, a.q_scale, a.g, a.M, a.K};
    adapters_da_kernel<T, C><<<dim3(blocks_of(a.K, kB), ry, L), kThreads, 0, st>>>(sum, in, static_cast<T*>(a.da), a.K,
                                                                                  R, a.plan);
    adapters_db_kernel<T, C><<<dim3(blocks_of(a.N, kB), ry, L), kThreads, 0, st>>>(
        static_cast<const T*>(a.dy), a.u, a.scales, static_cast<T*>(a.db), a.N, R, a.plan);
    return cudaGetLastError();
}

template <typename T>
cudaError_t forward_t(const AdapterFwdArgs& a, cudaStream_t st)
{
    return a.R <= 16 ? forward_c<T, 1>(a, st) : a.R <= 32 ? forward_c<T, 2>(a, st) : forward_c<T, 4>(a, st);
}
template <typename T>
cudaError_t backward_t(const AdapterBwdArgs& a, cudaStream_t st)
{
    return a.R <= 16 ? backward_c<T, 1>(a, st) : a.R <= 32 ? backward_c<T, 2>(a, st) : backward_c<T, 4>(a, st);
}

}  // namespace

cudaError_t launch_adapters_plan(const int32_t* ids, int64_t M, int64_t L, void* plan, cudaStream_t st)
{
    const int smem = (int)(32 * (L + 1) * sizeof(int));
    const cudaError_t e = allow_launch(reinterpret_cast<const void*>(adapters_plan_kernel), smem);
    if (e != cudaSuccess)
        return e;
    adapters_plan_kernel<<<1, 1024, smem, st>>>(ids, (int)M, (int)L, plan_view(plan, M, L));
    return cudaGetLastError();
}

size_t adapters_simt_workspace(int64_t M, int64_t N, int64_t K, int64_t R)
{
    return (size_t)(parts_of(K > N ? K : N) + 1) * (size_t)M * (size_t)R * sizeof(float);
}

cudaError_t launch_adapters_forward_simt(const AdapterFwdArgs& a, cudaStream_t st)
{
    return a.dt == QLIN_F32    ? forward_t<float>(a, st)
           : a.dt == QLIN_BF16 ? forward_t<__nv_bfloat16>(a, st)
                               : forward_t<__half>(a, st);
}

cudaError_t launch_adapters_backward_simt(const AdapterBwdArgs& a, cudaStream_t st)
{
    return a.dt == QLIN_F32    ? backward_t<float>(a, st)
           : a.dt == QLIN_BF16 ? backward_t<__nv_bfloat16>(a, st)
                               : backward_t<__half>(a, st);
}

}  // namespace qlin
