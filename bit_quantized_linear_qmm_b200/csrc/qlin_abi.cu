// qlin_abi.cu -- the extern "C" boundary of libqlin.so: argument validation,
// device checks, workspace sizing and dispatch to the kernel launchers.
// No exception crosses this file's functions; every failure is a qlin_status.
#include <initializer_list>
#include <mutex>

#include "adapters.cuh"
#include "qlin_common.cuh"

namespace qlin {

// Device status word: kernels OR kStatusTimeout into it when a bounded wait
// gives up; qlin_get_device_status() reads and clears it.
__device__ unsigned g_device_status;

// k_quant.cu: the per-row int8 quantiser launched as a programmatic dependent of the stream's
// previous kernel (its CTAs may be placed early and wait before touching memory); it also lets
// the next kernel start its prologue early.
cudaError_t launch_quantize_int8_rows_dependent(const void* w, qlin_dtype w_dt, int64_t R, int64_t C, int8_t* q,
                                                float* scale, cudaStream_t st, const DeviceInfo& dev);
// k_tc_gemm.cu: the CTA tile of the int8 tcgen05 GEMM, mt sub-tiles of 128 tokens by bn columns.
void tc_tile_shape(TcOp op, int64_t M, int64_t N, int64_t sms, int& mt, int& bn);

// k_checkpoint.cu
cudaError_t launch_dequantize_int8_groups(const int8_t* q, const float* scale, int64_t N, int64_t K, int g, void* out,
                                          qlin_dtype o_dt, cudaStream_t st);
cudaError_t launch_pergroup_wgrad(const void* dy, qlin_dtype dt, int64_t M, int64_t N, const int8_t* q,
                                  const float* scale, int64_t K, int g, void* dw, void* db, cudaStream_t st,
                                  const DeviceInfo& dev);

namespace {

constexpr int kMaxDevices = 64;

struct DeviceSlot {
    std::once_flag once;
    qlin_status state = QLIN_ERR_DEVICE;
    DeviceInfo info = {0, nullptr};
};

DeviceSlot g_slots[kMaxDevices];

}  // namespace

// Checks (once per device) that the current device is an sm_100 part, and
// records its SM count and the address of the status word.  Must run with
// that device current, outside stream capture (the first call per device).
qlin_status current_device(DeviceInfo& out)
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return QLIN_ERR_DEVICE;
    }
    DeviceSlot& slot = g_slots[dev];
    std::call_once(slot.once, [&slot, dev]() {
        cudaDeviceProp prop;
        if (cudaGetDeviceProperties(&prop, dev) != cudaSuccess) {
            cudaGetLastError();
            slot.state = QLIN_ERR_DEVICE;
            return;
        }
        if (prop.major != 10 || prop.minor != 0) {
            slot.state = QLIN_ERR_DEVICE;
            return;
        }
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_status) != cudaSuccess || p == nullptr) {
            cudaGetLastError();
            slot.state = QLIN_ERR_CUDA;
            return;
        }
        slot.info.sm_count = prop.multiProcessorCount;
        slot.info.status = static_cast<unsigned*>(p);
        slot.state = QLIN_OK;
    });
    out = slot.info;
    return slot.state;
}

cudaError_t allow_launch(const void* kern, int smem, bool wide)
{
    // every kernel has 48 KB less its static shared memory, which is not known here: 24 KB are safe
    if (smem <= 24 * 1024 && !wide)
        return cudaSuccess;
    struct Entry {
        const void* kern;
        int dev, smem;
        bool wide;
    };
    constexpr unsigned kEntries = 4096;  // kernels of the library x devices; without a free one: set each time
    static Entry entries[kEntries];
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned first = (unsigned)((reinterpret_cast<uintptr_t>(kern) >> 4) * 31u + (unsigned)dev);
    std::lock_guard<std::mutex> lock(mu);
    Entry* at = nullptr;
    for (unsigned i = 0; i < kEntries && !at; ++i) {
        Entry& s = entries[(first + i) % kEntries];
        if (!s.kern || (s.kern == kern && s.dev == dev))
            at = &s;
    }
    const bool known = at && at->kern;
    int had = known ? at->smem : 0;
    if (!at) {
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess)
            return e;
        had = fa.maxDynamicSharedSizeBytes;
    }
    const bool had_wide = known && at->wide;
    if (smem > had && (e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
        return e;
    if (wide && !had_wide &&
        (e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
        return e;
    if (at)
        *at = {kern, dev, smem > had ? smem : had, wide || had_wide};
    return cudaSuccess;
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool dtype_ok(qlin_dtype d) { return d == QLIN_F32 || d == QLIN_BF16 || d == QLIN_F16; }
size_t dtype_size(qlin_dtype d) { return d == QLIN_F32 ? 4 : 2; }
bool bits_ok(int b) { return (b >= 1 && b <= 6) || b == 8; }
bool group_ok(int g) { return g == 32 || g == 64 || g == 128; }
size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

qlin_status from_cuda(cudaError_t e)
{
    if (e == cudaSuccess)
        return QLIN_OK;
    cudaGetLastError();  // clear a non-sticky launch error
    return e == cudaErrorNotSupported ? QLIN_ERR_UNSUPPORTED : QLIN_ERR_CUDA;
}

bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
bool int8_group_ok(int g) { return g == 64 || g == 128 || g == 256; }
constexpr int64_t kMaxFeatures = 1 << 21;  // K, N of the adapter calls and of wgrad: block counts of a grid
// Tokens of a weight gradient: fp32 sums of as many terms of one size still grow, and a tile of them (1.44
// us a stage of 64) takes 0.4 s, where a wait for its sums gives up after 2 s.
constexpr int64_t kMaxWgradTokens = 1 << 24;

// Sizes of the adapter calls: INVALID_ARG below 1, UNSUPPORTED above what the kernels hold.
qlin_status check_plan(int64_t M, int64_t L)
{
    if (M <= 0 || L <= 0)
        return QLIN_ERR_INVALID_ARG;
    return M <= kMaxPlanTokens && L <= kMaxAdapters ? QLIN_OK : QLIN_ERR_UNSUPPORTED;
}
qlin_status check_adapters(qlin_dtype dt, int64_t M, int64_t N, int64_t K, int64_t L, int64_t R, const void* plan,
                           size_t plan_bytes)
{
    if (N <= 0 || K <= 0 || R <= 0)
        return QLIN_ERR_INVALID_ARG;
    const qlin_status s = check_plan(M, L);
    if (s != QLIN_OK)
        return s;
    if (!dtype_ok(dt) || R > kMaxRank || N >= kMaxFeatures || K >= kMaxFeatures)
        return QLIN_ERR_UNSUPPORTED;
    if (plan_bytes < qlin_adapters_plan_size(M, L))
        return QLIN_ERR_INVALID_ARG;
    return aligned16(plan) ? QLIN_OK : QLIN_ERR_MISALIGNED;
}

// Every non-null pointer is a multiple of `bytes`.
template <typename... P>
bool aligned_to(size_t bytes, const P*... p)
{
    return (((reinterpret_cast<uintptr_t>(p) % bytes) | ...) == 0);
}
bool overlap(const void* p, size_t pn, const void* q, size_t qn)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && a < b + qn && b < a + pn;
}
struct Span {
    const void* p;  // null: not given
    size_t n;
};
// Nothing that a call writes lies over anything it reads, or over anything else it writes.
bool apart(std::initializer_list<Span> written, std::initializer_list<Span> read)
{
    for (const Span* w = written.begin(); w != written.end(); ++w) {
        for (const Span* o = written.begin(); o != w; ++o)
            if (overlap(w->p, w->n, o->p, o->n))
                return false;
        for (const Span& r : read)
            if (overlap(w->p, w->n, r.p, r.n))
                return false;
    }
    return true;
}

// Shape/type rules common to the affine-format calls.
qlin_status check_affine(int64_t N, int64_t K, int bits, int g, qlin_dtype p_dt)
{
    if (N <= 0 || K <= 0 || N > INT32_MAX || K > INT32_MAX)
        return QLIN_ERR_INVALID_ARG;
    if (!bits_ok(bits) || !group_ok(g) || !dtype_ok(p_dt))
        return QLIN_ERR_UNSUPPORTED;
    if (K % g != 0)
        return QLIN_ERR_INVALID_ARG;
    return QLIN_OK;
}

}  // namespace
}  // namespace qlin

using namespace qlin;

namespace qlin {
// self-test of the bounded-wait path (k_selftest.cu): one wait that runs out after limit_ns.
cudaError_t launch_wait_timeout_selftest(unsigned long long limit_ns, cudaStream_t st, const DeviceInfo& dev);
}  // namespace qlin

extern "C" {

const char* qlin_status_string(qlin_status s)
{
    switch (s) {
    case QLIN_OK: return "QLIN_OK";
    case QLIN_ERR_INVALID_ARG: return "QLIN_ERR_INVALID_ARG: invalid argument";
    case QLIN_ERR_UNSUPPORTED: return "QLIN_ERR_UNSUPPORTED: unsupported bits/group/dtype combination";
    case QLIN_ERR_MISALIGNED: return "QLIN_ERR_MISALIGNED: pointer or row pitch not 16-byte aligned";
    case QLIN_ERR_DEVICE: return "QLIN_ERR_DEVICE: no sm_100 CUDA device current";
    case QLIN_ERR_CUDA: return "QLIN_ERR_CUDA: CUDA runtime error";
    case QLIN_ERR_TIMEOUT: return "QLIN_ERR_TIMEOUT: a bounded device wait expired";
    case QLIN_ERR_WORKSPACE: return "QLIN_ERR_WORKSPACE: workspace missing or too small";
    }
    return "QLIN_ERR_?: unknown status";
}

int qlin_version(void) { return 1 * 10000 + 0 * 100 + 0; }

qlin_status qlin_int8_gemm_tile(qlin_op op, int64_t M, int64_t N, int sm_count, int* tokens, int* columns)
{
    if ((op != QLIN_OP_W8A8 && op != QLIN_OP_W4A8) || M < 1 || N < 1 || sm_count < 1 || !tokens || !columns)
        return QLIN_ERR_INVALID_ARG;
    int mt = 1, bn = 256;
    tc_tile_shape(op == QLIN_OP_W4A8 ? TC_W4A8 : TC_W8A8, M, N, sm_count, mt, bn);
    *tokens = 128 * mt;
    *columns = bn;
    return QLIN_OK;
}

size_t qlin_workspace_size(qlin_op op, int64_t M, int64_t N, int64_t K, int bits, int group_size)
{
    if (M <= 0 || K <= 0)
        return 0;
    switch (op) {
    case QLIN_OP_W8A8:
    case QLIN_OP_W4A8: return align256((size_t)M * (size_t)K) + align256((size_t)M * 4);
    case QLIN_OP_PERGROUP:
        return (N > 0 && (group_size == 64 || group_size == 128 || group_size == 256) && K % group_size == 0)
                   ? tc_affine_workspace(M, N, K, group_size)
                   : 0;
    case QLIN_OP_MATMUL:
        // the tensor-core prefill (M > 16, 4-bit codes): fp16 x and group parameters, scales
        return (M > 16 && bits == 4 && N > 0 && group_size > 0 && K % group_size == 0)
                   ? tc_affine_workspace(M, N, K, group_size)
                   : 0;
    default: return 0;
    }
}

qlin_status qlin_quantize(const void* w, qlin_dtype w_dt, int64_t N, int64_t K, int bits, int group_size,
                          uint32_t* codes, void* scales, void* biases, qlin_dtype param_dt, void* stream)
{
    if (!w || !codes || !scales || !biases)
        return QLIN_ERR_INVALID_ARG;
    if (!dtype_ok(w_dt))
        return QLIN_ERR_UNSUPPORTED;
    qlin_status s = check_affine(N, K, bits, group_size, param_dt);
    if (s != QLIN_OK)
        return s;
    DeviceInfo dev;
    if ((s = current_device(dev)) != QLIN_OK)
        return s;
    return from_cuda(launch_affine_quantize(w, w_dt, N, K, bits, group_size, codes, scales, biases, param_dt,
                                            static_cast<cudaStream_t>(stream), dev));
}

qlin_status qlin_dequantize(const uint32_t* codes, const void* scales, const void* biases, qlin_dtype param_dt,
                            int64_t N, int64_t K, int bits, int group_size, void* w_out, qlin_dtype out_dt,
                            void* stream)
{
    if (!codes || !scales || !biases || !w_out)
        return QLIN_ERR_INVALID_ARG;
    if (!dtype_ok(out_dt))
        return QLIN_ERR_UNSUPPORTED;
    qlin_status s = check_affine(N, K, bits, group_size, param_dt);
    if (s != QLIN_OK)
        return s;
    // one word's outputs go out as 8- or 16-byte vector stores
    if (!aligned16(w_out) || (reinterpret_cast<uintptr_t>(codes) & 3u) != 0)
        return QLIN_ERR_MISALIGNED;
    DeviceInfo dev;
    if ((s = current_device(dev)) != QLIN_OK)
        return s;
    return from_cuda(launch_affine_dequantize(codes, scales, biases, param_dt, N, K, bits, group_size, w_out, out_dt,
                                              static_cast<cudaStream_t>(stream), dev));
}

qlin_status qlin_matmul(const void* x, qlin_dtype x_dt, int64_t M, int64_t K, const uint32_t* codes,
                        const void* scales, const void* biases, qlin_dtype param_dt, int64_t N, int bits,
                        int group_size, const void* bias, void* y, void* workspace, size_t ws_bytes, void* stream)
{
    if (!x || !codes || !scales || !biases || !y || M <= 0 || M > INT32_MAX)
        return QLIN_ERR_INVALID_ARG;
    if (!dtype_ok(x_dt))
        return QLIN_ERR_UNSUPPORTED;
    qlin_status s = check_affine(N, K, bits, group_size, param_dt);
    if (s != QLIN_OK)
        return s;
    // the specialized paths: power-of-two widths (not 2 bits in groups of 32), fp32 / bf16 operands,
    // TMA-loaded rows (16-byte pitch); the tensor-core prefill also takes fp16 x.  Everything else
    // runs the general decode kernel, which needs 4-byte aligned codes and 16-byte x rows.
    const bool tma_rows = aligned16(codes) && (K * bits / 8) % 16 == 0;
    const bool prefill = M > 16 && bits == 4 && param_dt == QLIN_BF16 && tma_rows;
    const bool special = (bits == 2 || bits == 4 || bits == 8) && !(bits == 2 && group_size == 32) &&
                         x_dt != QLIN_F16 && param_dt != QLIN_F16 && tma_rows;
    if (!aligned16(x) || (K * (int64_t)dtype_size(x_dt)) % 16 != 0 || (reinterpret_cast<uintptr_t>(codes) & 3u) != 0)
        return QLIN_ERR_MISALIGNED;
    DeviceInfo dev;
    if ((s = current_device(dev)) != QLIN_OK)
        return s;
    if (prefill) {
        const size_t need = qlin_workspace_size(QLIN_OP_MATMUL, M, N, K, bits, group_size);
        if (!workspace || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
            return QLIN_ERR_WORKSPACE;
        TcGemmArgs t = {};
        t.M = M;
        t.N = N;
        t.K = K;
        t.a = x;
        t.b = codes;
        t.out = y;
        t.bias = bias;
        t.scales = scales;
        t.biases = biases;
        t.g = group_size;
        t.bits = bits;
        t.x_dt = x_dt;
        t.workspace = workspace;
        return from_cuda(launch_tc_affine(t, static_cast<cudaStream_t>(stream), dev));
    }
    AffineGemvArgs a;
    a.x = x;
    a.x_dt = x_dt;
    a.M = M;
    a.K = K;
    a.N = N;
    a.codes = codes;
    a.scales = scales;
    a.biases = biases;
    a.p_dt = param_dt;
    a.bits = bits;
    a.g = group_size;
    a.bias = bias;
    a.y = y;
    return from_cuda(special ? launch_affine_gemv(a, static_cast<cudaStream_t>(stream), dev)
                             : launch_affine_gemv_any(a, static_cast<cudaStream_t>(stream), dev));
}

qlin_status bitlinear_matmul(const void* x, qlin_dtype x_dt, int64_t M, int64_t K, const uint8_t* packed, int64_t N,
                             const float* weight_scale, int invert_weight_scale, const void* bias, void* y,
                             void* stream)
{
    if (!x || !packed || !weight_scale || !y || M <= 0 || K <= 0 || N <= 0 || M > INT32_MAX || K > INT32_MAX ||
        N > INT32_MAX)
        return QLIN_ERR_INVALID_ARG;
    if (N % 4 != 0 || K % 16 != 0)
        return QLIN_ERR_INVALID_ARG;
    if (x_dt != QLIN_BF16)
        return QLIN_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(packed))
        return QLIN_ERR_MISALIGNED;
    DeviceInfo dev;
    qlin_status s;
    if ((s = current_device(dev)) != QLIN_OK)
        return s;
    BitlinearArgs a;
    a.x = x;
    a.x_dt = x_dt;
    a.M = M;
    a.K = K;
    a.N = N;
    a.packed = packed;
    a.weight_scale = weight_scale;
    a.invert = invert_weight_scale ? 1 : 0;
    a.bias = bias;
    a.y = y;
    if (M > 16)  // prefill: the tcgen05 GEMM reads the packed weights once per 256-token tile
        return from_cuda(launch_tc_bitlinear(a, static_cast<cudaStream_t>(stream), dev));
    return from_cuda(launch_bitlinear_gemv(a, static_cast<cudaStream_t>(stream), dev));
}

qlin_status qlin_quantize_int8_rows(const void* w, qlin_dtype w_dt, int64_t R, int64_t C, int8_t* q, float* scale,
                                    void* stream)
{
    if (!w || !q || !scale || R <= 0 || C <= 0 || R > INT32_MAX)
        return QLIN_ERR_INVALID_ARG;
    if (!dtype_ok(w_dt))
        return QLIN_ERR_UNSUPPORTED;
    DeviceInfo dev;
    qlin_status s;
    if ((s = current_device(dev)) != QLIN_OK)
        return s;
    return from_cuda(
        launch_quantize_int8_rows(w, w_dt, R, C, q, scale, static_cast<cudaStream_t>(stream), dev));
}

qlin_status qlin_pack_int4_cols(const void* w, qlin_dtype w_dt, int64_t K, int64_t N, uint8_t* packed, float* scale,
                                void* stream)
{
    if (!w || !packed || !scale || K <= 0 || N <= 0 || K % 2 != 0 || N > INT32_MAX)
        return QLIN_ERR_INVALID_ARG;
    if (!dtype_ok(w_dt))
        return QLIN_ERR_UNSUPPORTED;
    DeviceInfo dev;
    qlin_status s;
    if ((s = current_device(dev)) != QLIN_OK)
        return s;
    return from_cuda(launch_pack_int4_cols(w, w_dt, K, N, packed, scale, static_cast<cudaStream_t>(stream), dev));
}

qlin_status qlin_quantize_weight_int8(const void* w, qlin_dtype w_dt, int64_t R, int64_t C, double clip_percentile,
                                     int8_t* q, float* scale, void* stream)
{
    if (!w || !q || !scale || R <= 0 || C <= 0 || R > INT32_MAX || C > INT32_MAX)
        return QLIN_ERR_INVALID_ARG;
    if (!dtype_ok(w_dt))
        return QLIN_ERR_UNSUPPORTED;
    if (clip_percentile > 100.0 || clip_percentile != clip_percentile)
        return QLIN_ERR_INVALID_ARG;
    DeviceInfo dev;
    qlin_status s;
    if ((s = current_device(dev)) != QLIN_OK)
        return s;
    if (clip_percentile < 0.0)  // no clip: the absmax rule
        return from_cuda(
            launch_quantize_int8_rows(w, w_dt, R, C, q, scale, static_cast<cudaStream_t>(stream), dev));
    if (C > 32768)  // the row is held in shared memory
        return QLIN_ERR_UNSUPPORTED;
    // numpy converts the percentile to the row's float32 before dividing by 100
    return from_cuda(launch_quantize_weight_int8_clip(w, w_dt, R, C, (float)clip_percentile, q, scale,
                                                      static_cast<cudaStream_t>(stream), dev));
}

qlin_status qlin_quantize_int8_groups(const void* w, qlin_dtype w_dt, int64_t N, int64_t K, int group_size,
                                     int8_t* q, float* scale_w, void* stream)
{
    if (!w || !q || !scale_w || N <= 0 || K <= 0 || N > INT32_MAX || K > INT32_MAX)
        return QLIN_ERR_INVALID_ARG;
    if (!dtype_ok(w_dt) || !(group_size == 64 || group_size == 128 || group_size == 256))
        return QLIN_ERR_UNSUPPORTED;
    if (K % group_size != 0)
        return QLIN_ERR_INVALID_ARG;
    DeviceInfo dev;
    qlin_status s;
    if ((s = current_device(dev)) != QLIN_OK)
        return s;
    return from_cuda(
        launch_quantize_int8_groups(w, w_dt, N, K, group_size, q, scale_w, static_cast<cudaStream_t>(stream), dev));
}

qlin_status pergroup_linear(const void* x, qlin_dtype x_dt, int64_t M, int64_t K, const int8_t* w,
                            const float* scale_w, int64_t N, int group_size, const void* bias, void* y,
                            void* workspace, size_t ws_bytes, void* stream)
{
    if (!x || !w || !scale_w || !y || M <= 0 || N <= 0 || K <= 0 || M > INT32_MAX || N > INT32_MAX ||
        K > INT32_MAX)
        return QLIN_ERR_INVALID_ARG;
    if (!dtype_ok(x_dt) || !(group_size == 64 || group_size == 128 || group_size == 256))
        return QLIN_ERR_UNSUPPORTED;
    if (K % group_size != 0)
        return QLIN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w) || K % 16 != 0)
        return QLIN_ERR_MISALIGNED;
    const size_t need = qlin_workspace_size(QLIN_OP_PERGROUP, M, N, K, 8, group_size);
    if (!workspace || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return QLIN_ERR_WORKSPACE;
    DeviceInfo dev;
    qlin_status s;
    if ((s = current_device(dev)) != QLIN_OK)
        return s;
    if (M == 1 && x_dt == QLIN_BF16) {  // the FP-activation branch as a weight-resident decode GEMV
        AffineGemvArgs a;
        a.x = x;
        a.x_dt = x_dt;
        a.M = M;
        a.K = K;
        a.N = N;
        a.codes = reinterpret_cast<const uint32_t*>(w);
        a.scales = scale_w;
        a.biases = scale_w;  // not read
        a.p_dt = QLIN_F32;
        a.bits = 8;
        a.g = group_size;
        a.bias = bias;
        a.y = y;
        a.pergroup = 1;
        const cudaError_t e = launch_affine_dec(a, static_cast<cudaStream_t>(stream), dev);
        if (e != cudaErrorNotSupported)
            return from_cuda(e);
    }
    TcGemmArgs t = {};
    t.M = M;
    t.N = N;
    t.K = K;
    t.a = x;
    t.b = w;
    t.out = y;
    t.bias = bias;
    t.scales = scale_w;
    t.biases = nullptr;
    t.g = group_size;
    t.bits = 8;
    t.x_dt = x_dt;
    t.pergroup = 1;
    t.workspace = workspace;
    return from_cuda(launch_tc_affine(t, static_cast<cudaStream_t>(stream), dev));
}

qlin_status qlin_int8_matmul_int32(const int8_t* a, const int8_t* b, int64_t M, int64_t N, int64_t K, int32_t* c,
                                   void* stream)
{
    if (!a || !b || !c || M <= 0 || N <= 0 || K <= 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX)
        return QLIN_ERR_INVALID_ARG;
    if (K % 16 != 0)
        return QLIN_ERR_INVALID_ARG;
    if (!aligned16(a) || !aligned16(b) || !aligned16(c))
        return QLIN_ERR_MISALIGNED;
    DeviceInfo dev;
    qlin_status s;
    if ((s = current_device(dev)) != QLIN_OK)
        return s;
    TcGemmArgs t = {};
    t.M = M;
    t.N = N;
    t.K = K;
    t.a = a;
    t.b = b;
    t.out = c;
    return from_cuda(launch_tc_gemm(TC_I8_RAW, t, static_cast<cudaStream_t>(stream), dev));
}

namespace {

// Shared body of the W8A8 / W4A8 layers: per-token int8 activation quant
// into the workspace, then the tcgen05 GEMM with the scaled epilogue.
qlin_status int_linear(TcOp op, const void* x, qlin_dtype x_dt, int64_t M, int64_t K, const void* w,
                       const float* scale_w, int64_t N, const void* bias, void* y, void* workspace, size_t ws_bytes,
                       void* stream)
{
    if (!x || !w || !scale_w || !y || M <= 0 || N <= 0 || K <= 0 || M > INT32_MAX || N > INT32_MAX ||
        K > INT32_MAX)
        return QLIN_ERR_INVALID_ARG;
    if (op == TC_W4A8 ? (K % 32 != 0 || N % 16 != 0) : (K % 16 != 0))
        return QLIN_ERR_INVALID_ARG;
    if (x_dt != QLIN_BF16 && x_dt != QLIN_F16)  // y and bias take x's 16-bit dtype
        return QLIN_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(w) || !aligned16(y))
        return QLIN_ERR_MISALIGNED;
    const size_t need = qlin_workspace_size(op == TC_W4A8 ? QLIN_OP_W4A8 : QLIN_OP_W8A8, M, N, K, 0, 0);
    if (!workspace || ws_bytes < need || !aligned16(workspace))
        return QLIN_ERR_WORKSPACE;
    DeviceInfo dev;
    qlin_status s;
    if ((s = current_device(dev)) != QLIN_OK)
        return s;
    int8_t* qx = static_cast<int8_t*>(workspace);
    float* sx = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align256((size_t)M * (size_t)K));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // the quantiser lets the next kernel start its prologue (fetching the layer's weights) early;
    // ahead of a tcgen05 GEMM it is also placed early itself, behind the stream's previous kernel
    cudaError_t e = M > 16 ? launch_quantize_int8_rows_dependent(x, x_dt, M, K, qx, sx, st, dev)
                           : launch_quantize_int8_rows(x, x_dt, M, K, qx, sx, st, dev, true);
    if (e != cudaSuccess)
        return from_cuda(e);
    if (M <= 16) {  // decode: weight-streaming GEMV on int8 mma.sync
        W8GemvArgs g;
        g.qx = qx;
        g.s_x = sx;
        g.w = static_cast<const int8_t*>(w);
        g.s_w = scale_w;
        g.bias = bias;
        g.y = y;
        g.M = M;
        g.K = K;
        g.N = N;
        g.out_f16 = x_dt == QLIN_F16;
        return from_cuda(op == TC_W8A8 ? launch_w8_gemv(g, st, dev) : launch_w4_gemv(g, st, dev));
    }
    TcGemmArgs t = {};
    t.M = M;
    t.N = N;
    t.K = K;
    t.a = qx;
    t.b = w;
    t.out = y;
    t.s_x = sx;
    t.s_w = scale_w;
    t.bias = bias;
    t.x_dt = x_dt;
    return from_cuda(launch_tc_gemm(op, t, st, dev));
}

}  // namespace

qlin_status w8a8_linear(const void* x, qlin_dtype x_dt, int64_t M, int64_t K, const int8_t* w, const float* scale_w,
                        int64_t N, const void* bias, void* y, void* workspace, size_t ws_bytes, void* stream)
{
    return int_linear(TC_W8A8, x, x_dt, M, K, w, scale_w, N, bias, y, workspace, ws_bytes, stream);
}

qlin_status w4a8_linear(const void* x, qlin_dtype x_dt, int64_t M, int64_t K, const uint8_t* packed_w,
                        const float* scale_w, int64_t N, const void* bias, void* y, void* workspace, size_t ws_bytes,
                        void* stream)
{
    return int_linear(TC_W4A8, x, x_dt, M, K, packed_w, scale_w, N, bias, y, workspace, ws_bytes, stream);
}

size_t qlin_adapters_plan_size(int64_t M, int64_t L)
{
    return check_plan(M, L) == QLIN_OK ? align256((size_t)plan_ints(M, L) * sizeof(int)) : 0;
}

qlin_status qlin_adapters_plan(const int32_t* ids, int64_t M, int64_t L, void* plan, size_t plan_bytes, void* stream)
{
    if (!ids || !plan)
        return QLIN_ERR_INVALID_ARG;
    qlin_status s = check_plan(M, L);
    if (s != QLIN_OK)
        return s;
    if (plan_bytes < qlin_adapters_plan_size(M, L))
        return QLIN_ERR_INVALID_ARG;
    if (!aligned16(plan) || (reinterpret_cast<uintptr_t>(ids) & 3u) != 0)
        return QLIN_ERR_MISALIGNED;
    DeviceInfo dev;
    if ((s = current_device(dev)) != QLIN_OK)
        return s;
    if (!apart({{plan, qlin_adapters_plan_size(M, L)}}, {{ids, (size_t)M * 4}}))
        return QLIN_ERR_INVALID_ARG;
    return from_cuda(launch_adapters_plan(ids, M, L, plan, static_cast<cudaStream_t>(stream)));
}

size_t qlin_adapters_workspace_size(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R, int)
{
    if (check_plan(M, L) != QLIN_OK || N <= 0 || K <= 0 || R <= 0 || R > kMaxRank || N >= kMaxFeatures ||
        K >= kMaxFeatures)
        return 0;
    const size_t simt = align256(adapters_simt_workspace(M, N, K, R)), tc = align256(adapters_tc_workspace(M, N, L, R));
    return simt > tc ? simt : tc;
}

qlin_status qlin_adapters_forward(const void* x, qlin_dtype dt, int64_t M, int64_t K, const void* a, const void* b,
                                  const float* scales, int64_t L, int64_t R, int64_t N, const void* plan,
                                  size_t plan_bytes, const void* base, void* out, float* u, void* workspace,
                                  size_t ws_bytes, void* stream)
{
    if (!x || !a || !b || !scales || !plan || !out)
        return QLIN_ERR_INVALID_ARG;
    qlin_status s = check_adapters(dt, M, N, K, L, R, plan, plan_bytes);
    if (s != QLIN_OK)
        return s;
    const size_t e = dtype_size(dt), on = M * N * e, ws_need = qlin_adapters_workspace_size(M, N, K, L, R, 0);
    if (!aligned_to(e, x, a, b, base, out) || !aligned_to(4, scales, u))
        return QLIN_ERR_MISALIGNED;
    const Span out_s = {out, on}, u_s = {u, (size_t)(M * R) * 4}, x_s = {x, M * K * e}, a_s = {a, L * R * K * e},
               b_s = {b, L * N * R * e}, sc_s = {scales, (size_t)L * 4}, base_s = {base == out ? nullptr : base, on},
               plan_s = {plan, qlin_adapters_plan_size(M, L)};
    if (!apart({out_s, u_s}, {x_s, a_s, b_s, sc_s, base_s, plan_s}))
        return QLIN_ERR_INVALID_ARG;
    if (!workspace || ws_bytes < ws_need || !aligned256(workspace))
        return QLIN_ERR_WORKSPACE;
    DeviceInfo dev;
    if ((s = current_device(dev)) != QLIN_OK)
        return s;
    if (!apart({{workspace, ws_need}}, {out_s, u_s, x_s, a_s, b_s, sc_s, base_s, plan_s}))
        return QLIN_ERR_INVALID_ARG;
    const AdapterFwdArgs f = {x, a, b, scales, base, out, u, dt, M, K, N, L, R, plan_view(plan, M, L), workspace};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return from_cuda(adapters_tc_takes(f) ? launch_adapters_forward_tc(f, st, dev) : launch_adapters_forward_simt(f, st));
}

qlin_status qlin_adapters_backward(const void* dy, qlin_dtype dt, int64_t M, int64_t N, const void* a, const void* b,
                                   const float* scales, int64_t L, int64_t R, int64_t K, const void* plan,
                                   size_t plan_bytes, const float* u, const void* x, const int8_t* q,
                                   const float* q_scale, int group_size, const void* dx_base, void* dx, void* da,
                                   void* db, void* workspace, size_t ws_bytes, void* stream)
{
    if (!dy || !a || !b || !scales || !plan || !u || !da || !db || !x == !q || (q && !q_scale) || (dx_base && !dx))
        return QLIN_ERR_INVALID_ARG;
    qlin_status s = check_adapters(dt, M, N, K, L, R, plan, plan_bytes);
    if (s != QLIN_OK)
        return s;
    if (q && !int8_group_ok(group_size))
        return QLIN_ERR_UNSUPPORTED;
    if (q && K % group_size != 0)
        return QLIN_ERR_INVALID_ARG;
    const size_t e = dtype_size(dt), xn = M * K * e, an = L * R * K * e, bn = L * N * R * e,
                 ws_need = qlin_adapters_workspace_size(M, N, K, L, R, 1);
    if (!aligned_to(e, dy, a, b, x, dx_base, dx, da, db) || !aligned_to(4, scales, u, q_scale))
        return QLIN_ERR_MISALIGNED;
    const Span dx_s = {dx, xn}, dy_s = {dy, M * N * e}, a_s = {a, an}, b_s = {b, bn}, sc_s = {scales, (size_t)L * 4},
               u_s = {u, (size_t)(M * R) * 4}, x_s = {x, xn}, q_s = {q, (size_t)(M * K)},
               qs_s = {q ? q_scale : nullptr, q ? (size_t)(K / group_size * M) * 4 : 0},
               base_s = {dx_base == dx ? nullptr : dx_base, xn}, plan_s = {plan, qlin_adapters_plan_size(M, L)};
    if (!apart({dx_s}, {dy_s, a_s, b_s, sc_s, u_s, x_s, q_s, qs_s, base_s, plan_s}))
        return QLIN_ERR_INVALID_ARG;
    if (!workspace || ws_bytes < ws_need || !aligned256(workspace))
        return QLIN_ERR_WORKSPACE;
    DeviceInfo dev;
    if ((s = current_device(dev)) != QLIN_OK)
        return s;
    if (!apart({{da, an}, {db, bn}, {workspace, ws_need}, dx_s},
               {dy_s, a_s, b_s, sc_s, u_s, x_s, q_s, qs_s, base_s, plan_s}))
        return QLIN_ERR_INVALID_ARG;
    const AdapterBwdArgs g = {dy, a,  b,  scales, u,  x, q, q_scale, group_size, dx_base,
                              dx, da, db, dt,     M,  K, N, L,       R,          plan_view(plan, M, L),
                              workspace};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return from_cuda(adapters_tc_takes(g) ? launch_adapters_backward_tc(g, st, dev)
                                          : launch_adapters_backward_simt(g, st));
}

qlin_status qlin_dequantize_int8_groups(const int8_t* q, const float* scale, int64_t N, int64_t K, int group_size,
                                        void* out, qlin_dtype out_dt, void* stream)
{
    if (!q || !scale || !out || N <= 0 || K <= 0 || N > INT32_MAX || K > INT32_MAX)
        return QLIN_ERR_INVALID_ARG;
    if (!dtype_ok(out_dt) || !int8_group_ok(group_size))
        return QLIN_ERR_UNSUPPORTED;
    if (K % group_size != 0)
        return QLIN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned_to(4, scale))
        return QLIN_ERR_MISALIGNED;
    DeviceInfo dev;
    qlin_status s;
    if ((s = current_device(dev)) != QLIN_OK)
        return s;
    if (!apart({{out, N * K * dtype_size(out_dt)}}, {{q, (size_t)(N * K)}, {scale, (size_t)(K / group_size * N) * 4}}))
        return QLIN_ERR_INVALID_ARG;
    return from_cuda(launch_dequantize_int8_groups(q, scale, N, K, group_size, out, out_dt,
                                                   static_cast<cudaStream_t>(stream)));
}

qlin_status pergroup_wgrad(const void* dy, qlin_dtype dt, int64_t M, int64_t N, const int8_t* q, const float* scale,
                           int64_t K, int group_size, void* dw, void* db, void* stream)
{
    if (!dy || !q || !scale || !dw || M <= 0 || N <= 0 || K <= 0 || M > INT32_MAX)
        return QLIN_ERR_INVALID_ARG;
    if ((dt != QLIN_BF16 && dt != QLIN_F16) || !int8_group_ok(group_size) || N >= kMaxFeatures || K >= kMaxFeatures ||
        M > kMaxWgradTokens)
        return QLIN_ERR_UNSUPPORTED;
    if (K % group_size != 0)
        return QLIN_ERR_INVALID_ARG;
    if (N % 8 != 0 || !aligned16(dy) || !aligned16(q) || !aligned16(dw) || !aligned_to(4, scale) ||
        !aligned_to(2, db))
        return QLIN_ERR_MISALIGNED;
    DeviceInfo dev;
    qlin_status s;
    if ((s = current_device(dev)) != QLIN_OK)
        return s;
    if (!apart({{dw, (size_t)(N * K) * 2}, {db, (size_t)N * 2}},
               {{dy, (size_t)(M * N) * 2}, {q, (size_t)(M * K)}, {scale, (size_t)(K / group_size * M) * 4}}))
        return QLIN_ERR_INVALID_ARG;
    return from_cuda(launch_pergroup_wgrad(dy, dt, M, N, q, scale, K, group_size, dw, db,
                                           static_cast<cudaStream_t>(stream), dev));
}

qlin_status qlin_selftest_wait_timeout(unsigned limit_us, void* stream)
{
    if (limit_us == 0 || limit_us > 2000000u)
        return QLIN_ERR_INVALID_ARG;
    DeviceInfo dev;
    qlin_status s = current_device(dev);
    if (s != QLIN_OK)
        return s;
    return from_cuda(launch_wait_timeout_selftest((unsigned long long)limit_us * 1000ull,
                                                  static_cast<cudaStream_t>(stream), dev));
}

qlin_status qlin_get_device_status(void* stream)
{
    DeviceInfo dev;
    qlin_status s = current_device(dev);
    if (s != QLIN_OK)
        return s;
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        cudaGetLastError();
        return QLIN_ERR_CUDA;
    }
    unsigned word = 0;
    if (cudaMemcpy(&word, dev.status, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess) {
        cudaGetLastError();
        return QLIN_ERR_CUDA;
    }
    if (word != 0) {
        const unsigned zero = 0;
        cudaMemcpy(dev.status, &zero, sizeof(zero), cudaMemcpyHostToDevice);
        return QLIN_ERR_TIMEOUT;
    }
    return QLIN_OK;
}

}  // extern "C"

// ---------------------------------------------------------------- tensor maps (host)
#include <cudaTypedefs.h>

namespace qlin {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, []() {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        else
            cudaGetLastError();
    });
    return fn;
}

}  // namespace

bool encode_tmap_2d(CUtensorMap* tm, CUtensorMapDataType dt, const void* base, uint64_t dim0, uint64_t dim1,
                    uint64_t pitch_bytes, uint32_t box0, uint32_t box1, CUtensorMapSwizzle swizzle)
{
    const PFN_cuTensorMapEncodeTiled_v12000 fn = tmap_encoder();
    if (!fn)
        return false;
    cuuint64_t dims[2] = {dim0, dim1};
    cuuint64_t strides[1] = {pitch_bytes};
    cuuint32_t box[2] = {box0, box1};
    cuuint32_t estr[2] = {1, 1};
    return fn(tm, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_tmap_3d(CUtensorMap* tm, CUtensorMapDataType dt, const void* base, uint64_t dim0, uint64_t dim1,
                    uint64_t dim2, uint64_t elem_bytes, uint32_t box0, uint32_t box1)
{
    const PFN_cuTensorMapEncodeTiled_v12000 fn = tmap_encoder();
    if (!fn)
        return false;
    cuuint64_t dims[3] = {dim0, dim1, dim2};
    cuuint64_t strides[2] = {dim0 * elem_bytes, dim0 * dim1 * elem_bytes};
    cuuint32_t box[3] = {box0, box1, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(tm, dt, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace qlin
