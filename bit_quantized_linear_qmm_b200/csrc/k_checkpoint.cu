// k_checkpoint.cu -- activations kept in 8 bits for the backward pass: restoring them, and the
// weight gradient straight from them.
//
// A checkpoint of x [M tokens][K] is its per-group int8 quantisation (qlin_quantize_int8_groups):
// codes q [M][K] and fp32 scales [K/g][M] with x^[m][k] = q[m][k] scale[k/g][m].
//
//   restore   x^ in the type asked for
//   wgrad     dW[n][k] = sum_m dy[m][n] x^[m][k]      db[n] = sum_m dy[m][n]
#include "simt_tile.cuh"

namespace qlin {

cudaError_t launch_dequantize_int8_groups(const int8_t* q, const float* scale, int64_t N, int64_t K, int g, void* out,
                                          qlin_dtype o_dt, cudaStream_t st);
cudaError_t launch_pergroup_wgrad(const void* dy, qlin_dtype dt, int64_t M, int64_t N, const int8_t* q,
                                  const float* scale, int64_t K, int g, void* dw, void* db, cudaStream_t st,
                                  const DeviceInfo& dev);

namespace {

QLIN_DEV float code_of(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

// 16 codes a thread: one 16-byte load, one scale (a group is 64 codes at least), 16-byte stores.
// Memory-bound: 1 byte in and 2 or 4 out for each value.
template <typename T>
__global__ void __launch_bounds__(256) dequantize_int8_groups_kernel(const int8_t* __restrict__ q,
                                                                     const float* __restrict__ scale, int64_t N,
                                                                     int64_t K, int g_shift, T* __restrict__ out)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 16;
    if (i >= N * K)
        return;
    const int64_t n = i / K, grp = (i - n * K) >> g_shift;
    const uint4 v = ldg_stream_v4(q + i);
    const float s = __ldg(scale + grp * N + n);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<float4*>(out + i + 4 * j) =
                make_float4(code_of(w[j], 0) * s, code_of(w[j], 1) * s, code_of(w[j], 2) * s, code_of(w[j], 3) * s);
    } else {
        constexpr int f16 = sizeof(T) == 2 && !__is_same(T, __nv_bfloat16);
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h[2 * j] = pack_h16x2(code_of(w[j], 0) * s, code_of(w[j], 1) * s, f16);
            h[2 * j + 1] = pack_h16x2(code_of(w[j], 2) * s, code_of(w[j], 3) * s, f16);
        }
        *reinterpret_cast<uint4*>(out + i) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(out + i + 8) = make_uint4(h[4], h[5], h[6], h[7]);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) wgrad_kernel(const T* __restrict__ dy, const int8_t* __restrict__ q,
                                                         const float* __restrict__ scale, int64_t M, int64_t N,
                                                         int64_t K, int g_shift, T* __restrict__ dw)
{
    const int64_t n0 = (int64_t)blockIdx.x * kB, k0 = (int64_t)blockIdx.y * kB;
    float o[4][4];
    tile_product<false, false>(
        0, M, [&](int i, int64_t m) { return n0 + i < N ? to_float(dy[m * N + n0 + i]) : 0.f; },
        [&](int j, int64_t m) { return (float)q[m * K + k0 + j] * scale[((k0 + j) >> g_shift) * M + m]; }, o);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (n0 + 4 * ty + r < N)
                dw[(n0 + 4 * ty + r) * K + k0 + 4 * tx + c] = from_float<T>(o[r][c]);
}

template <typename T>
__global__ void __launch_bounds__(256) column_sum_kernel(const T* __restrict__ dy, int64_t M, int64_t N,
                                                         T* __restrict__ db)
{
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= N)
        return;
    float sum = 0.f;
    for (int64_t m0 = 0; m0 < M; m0 += kChunk) {
        float part = 0.f;
        for (int64_t m = m0; m < (m0 + kChunk < M ? m0 + kChunk : M); ++m)
            part += to_float(dy[m * N + n]);
        sum += part;
    }
    db[n] = from_float<T>(sum);
}

int log2_of(int g) { return g == 64 ? 6 : g == 128 ? 7 : 8; }

template <typename T>
cudaError_t wgrad_t(const T* dy, int64_t M, int64_t N, const int8_t* q, const float* scale, int64_t K, int g, T* dw,
                    T* db, cudaStream_t st)
{
    wgrad_kernel<T><<<dim3((unsigned)((N + kB - 1) / kB), (unsigned)(K / kB)), kThreads, 0, st>>>(
        dy, q, scale, M, N, K, log2_of(g), dw);
    if (db)
        column_sum_kernel<T><<<(unsigned)((N + 255) / 256), 256, 0, st>>>(dy, M, N, db);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dequantize_int8_groups(const int8_t* q, const float* scale, int64_t N, int64_t K, int g, void* out,
                                          qlin_dtype o_dt, cudaStream_t st)
{
    const unsigned blocks = (unsigned)((N * K / 16 + 255) / 256);
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
                                  const DeviceInfo&)
{
    if (dt == QLIN_BF16)
        return wgrad_t(static_cast<const __nv_bfloat16*>(dy), M, N, q, scale, K, g, static_cast<__nv_bfloat16*>(dw),
                       static_cast<__nv_bfloat16*>(db), st);
    return wgrad_t(static_cast<const __half*>(dy), M, N, q, scale, K, g, static_cast<__half*>(dw),
                   static_cast<__half*>(db), st);
}

}  // namespace qlin
