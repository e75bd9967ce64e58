// simt_tile.cuh -- a 64 x 16 C fp32 tile product on the CUDA cores, operands given by functors.
#pragma once

#include "qlin_common.cuh"

namespace qlin {

constexpr int kB = 64, kBK = 16, kThreads = 256, kChunk = 128;

// out[r][c] = sum over k in [k0, k1) of P(4 ty + r, k) Q(C tx + c, k), a tile of 64 by 16 C; P and Q
// return 0 outside their own ranges.  PK / QK: consecutive threads load consecutive k (rows of memory
// run along k).  The next 16 terms' operands are loaded while the last ones are multiplied.
template <int C, bool PK, bool QK, typename FP, typename FQ>
QLIN_DEV void tile_product(int64_t k0, int64_t k1, FP P, FQ Q, float (&out)[4][C])
{
    constexpr int W = 16 * C;
    __shared__ __align__(16) float ps[kBK][kB + 4], qs[kBK][W + 4];
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    float acc[4][C] = {};
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c)
            out[r][c] = 0.f;
    float p[4], q[C];
    auto load = [&](int64_t kb) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = tid + kThreads * j;
            const int64_t k = kb + (PK ? e % kBK : e / kB);
            p[j] = k < k1 ? P(PK ? e / kBK : e % kB, k) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int e = tid + kThreads * j;
            const int64_t k = kb + (QK ? e % kBK : e / W);
            q[j] = k < k1 ? Q(QK ? e / kBK : e % W, k) : 0.f;
        }
    };
    int64_t in_chunk = 0;
    if (k0 < k1)
        load(k0);
    for (int64_t kb = k0; kb < k1; kb += kBK) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = tid + kThreads * j;
            ps[PK ? e % kBK : e / kB][PK ? e / kBK : e % kB] = p[j];
        }
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int e = tid + kThreads * j;
            qs[QK ? e % kBK : e / W][QK ? e / kBK : e % W] = q[j];
        }
        __syncthreads();
        if (kb + kBK < k1)
            load(kb + kBK);
#pragma unroll
        for (int k = 0; k < kBK; ++k) {
            const float4 a = *reinterpret_cast<const float4*>(&ps[k][4 * ty]);
            const float av[4] = {a.x, a.y, a.z, a.w};
            float bv[C];
#pragma unroll
            for (int c = 0; c < C; ++c)
                bv[c] = qs[k][C * tx + c];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < C; ++c)
                    acc[r][c] = fmaf(av[r], bv[c], acc[r][c]);
        }
        in_chunk += kBK;
        if (in_chunk == kChunk || kb + kBK >= k1) {
            in_chunk = 0;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    out[r][c] += acc[r][c];
                    acc[r][c] = 0.f;
                }
        }
    }
}

}  // namespace qlin
