// simt_tile.cuh -- a 64 x 64 fp32 tile product on the CUDA cores, operands given by functors.
#pragma once

#include "qlin_common.cuh"

namespace qlin {

constexpr int kB = 64, kBK = 16, kThreads = 256, kChunk = 128;

// acc[r][c] = sum over k in [k0, k1) of P(4 ty + r, k) Q(4 tx + c, k); P and Q return 0 outside
// their own ranges.  PK / QK: consecutive threads load consecutive k (rows of memory run along k).
template <bool PK, bool QK, typename FP, typename FQ>
QLIN_DEV void tile_product(int64_t k0, int64_t k1, FP P, FQ Q, float (&out)[4][4])
{
    __shared__ __align__(16) float ps[kBK][kB + 4], qs[kBK][kB + 4];
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    float acc[4][4] = {};
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            out[r][c] = 0.f;
    int64_t in_chunk = 0;
    for (int64_t kb = k0; kb < k1; kb += kBK) {
        float p[4], q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = tid + kThreads * j;
            const int64_t pk = kb + (PK ? e % kBK : e / kB), qk = kb + (QK ? e % kBK : e / kB);
            p[j] = pk < k1 ? P(PK ? e / kBK : e % kB, pk) : 0.f;
            q[j] = qk < k1 ? Q(QK ? e / kBK : e % kB, qk) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = tid + kThreads * j;
            ps[PK ? e % kBK : e / kB][PK ? e / kBK : e % kB] = p[j];
            qs[QK ? e % kBK : e / kB][QK ? e / kBK : e % kB] = q[j];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kBK; ++k) {
            const float4 a = *reinterpret_cast<const float4*>(&ps[k][4 * ty]);
            const float4 b = *reinterpret_cast<const float4*>(&qs[k][4 * tx]);
            const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    acc[r][c] = fmaf(av[r], bv[c], acc[r][c]);
        }
        in_chunk += kBK;
        if (in_chunk == kChunk || kb + kBK >= k1) {
            in_chunk = 0;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    out[r][c] += acc[r][c];
                    acc[r][c] = 0.f;
                }
        }
    }
}

}  // namespace qlin
