// C ABI calls for what stands around a feed-forward block's GEMMs: the RMS norm, the products
// with 4-bit weights and dropout.  Argument checks and launches; nothing is kept between calls.
#include <atomic>
#include <cmath>
#include <initializer_list>

#include "plan.h"

using namespace gemm_epi;
using namespace gemm_epi_impl;

namespace {

bool is_16bit(gemm_epi_dtype dtype) { return dtype == GEMM_EPI_F16 || dtype == GEMM_EPI_BF16; }

// The current device's SM count once it is known to be an sm_103 device; the answer for a
// device never changes, so it is asked for once (these calls are made per token).
gemm_epi_status device_sms(int* sms)
{
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];
    int dev = -1;
    if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kDevices) {
        *sms = known[dev].load(std::memory_order_relaxed);
        if (*sms > 0) return GEMM_EPI_OK;
    }
    const gemm_epi_status st = current_device(sms);
    if (st == GEMM_EPI_OK && dev >= 0 && dev < kDevices)
        known[dev].store(*sms, std::memory_order_relaxed);
    return st;
}

gemm_epi_status launched(cudaError_t e) { return e == cudaSuccess ? GEMM_EPI_OK : GEMM_EPI_ERR_LAUNCH; }

// (widths to 2^30: the kernels step through them in 32 bits)
constexpr int64_t kMaxWidth = 1ll << 30;

bool norm_shape_ok(int64_t t, int64_t d)
{
    const int64_t kMax = (1ll << 31) - 1;
    return t >= 0 && d >= 8 && d % 8 == 0 && t <= kMax && d <= kMaxWidth && t * d <= (1ll << 40);
}

struct Buffer {
    const void* p;
    int64_t bytes;
};

bool meet(const Buffer& a, const Buffer& b)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x && y && x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}

// An output overlaps none of `others`, and those that it may be (of its own extent) not in part.
bool apart(const Buffer& out, std::initializer_list<Buffer> others, std::initializer_list<Buffer> may_be = {})
{
    for (const Buffer& b : others)
        if (meet(out, b)) return false;
    for (const Buffer& b : may_be)
        if (b.p != out.p && meet(out, b)) return false;
    return true;
}

int64_t round16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

gemm_epi_status rmsnorm(int64_t t, int64_t d, gemm_epi_dtype dtype, const void* X,
                        const void* residual, const void* gamma, float eps, void* H, void* Y,
                        int mode, float* scale, float* rstd, void* workspace, cudaStream_t stream)
{
    if (!is_16bit(dtype)) return GEMM_EPI_ERR_INVALID_ARG;
    if (!norm_shape_ok(t, d)) return GEMM_EPI_ERR_UNSUPPORTED_SHAPE;
    if (!(eps >= 0.0f) || !(eps < 1e30f)) return GEMM_EPI_ERR_INVALID_ARG;
    if (t == 0) return GEMM_EPI_OK;
    if (!X || !gamma || !Y || (residual != nullptr) != (H != nullptr) || H == Y)
        return GEMM_EPI_ERR_INVALID_ARG;
    if (mode != kRms16 && !scale) return GEMM_EPI_ERR_INVALID_ARG;
    if (mode != kRms16 && (Y == X || Y == residual)) return GEMM_EPI_ERR_INVALID_ARG;
    if (mode == kRmsTensor && !workspace) return GEMM_EPI_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(residual, 16) || !aligned(gamma, 16) || !aligned(H, 16) ||
        !aligned(Y, 16) || !aligned(scale, 4) || !aligned(rstd, 4) ||
        (mode == kRmsTensor && !aligned(workspace, 16)))
        return GEMM_EPI_ERR_MISALIGNED;
    {
        const Buffer x = {X, 2 * t * d}, r = {residual, 2 * t * d}, g = {gamma, 2 * d}, h = {H, 2 * t * d};
        const Buffer y = {Y, (mode == kRms16 ? 2 : 1) * t * d}, rs = {rstd, 4 * t};
        const Buffer sc = {scale, mode == kRmsRow ? 4 * t : 4};
        const Buffer ws = mode == kRmsTensor ? Buffer{workspace, gemm_epi_rmsnorm_workspace(t, d)} : Buffer{nullptr, 0};
        bool ok = apart(h, {g, y, rs}, {x, r}) && apart(rs, {x, r, g, y});
        if (mode == kRms16)
            ok = ok && apart(y, {g}, {x, r});
        else
            ok = ok && apart(y, {g, x, r, sc, ws}) && apart(sc, {h, rs, ws}) && apart(ws, {h, rs, x, r, g}) &&
                 (mode == kRmsGiven || apart(sc, {x, r, g}));
        if (!ok) return GEMM_EPI_ERR_INVALID_ARG;
    }
    int sms = 0;
    const gemm_epi_status st = device_sms(&sms);
    if (st != GEMM_EPI_OK) return st;
    RmsnormArgs a;
    a.X = X;
    a.residual = residual;
    a.gamma = gamma;
    a.H = H;
    a.Y = Y;
    a.scale = scale;
    a.rstd = rstd;
    a.ws_max = static_cast<uint32_t*>(workspace);
    a.ws_rstd = reinterpret_cast<float*>(a.ws_max + kRmsMaxParts);
    a.eps = eps;
    a.mode = mode;
    a.t = static_cast<int>(t);
    a.d = static_cast<int>(d);
    return launched(rmsnorm_launch(a, dtype == GEMM_EPI_BF16, stream));
}

gemm_epi_status w4_checked(int64_t n, int64_t k, int64_t group, gemm_epi_dtype dtype)
{
    if (!is_16bit(dtype)) return GEMM_EPI_ERR_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return GEMM_EPI_ERR_UNSUPPORTED_SHAPE;
    if (n < 0 || k < 0 || n > kMaxWidth || k > kMaxWidth || n % 8 != 0 || k % group != 0 || n * k > (1ll << 40))
        return GEMM_EPI_ERR_UNSUPPORTED_SHAPE;
    return GEMM_EPI_OK;
}

}  // namespace

extern "C" {

gemm_epi_status gemm_epi_rmsnorm(int64_t t, int64_t d, gemm_epi_dtype dtype, const void* X,
                                 const void* residual, const void* gamma, float eps, void* H,
                                 void* Y, float* rstd, cudaStream_t stream)
{
    return rmsnorm(t, d, dtype, X, residual, gamma, eps, H, Y, kRms16, nullptr, rstd, nullptr,
                   stream);
}

gemm_epi_status gemm_epi_rmsnorm_e4m3(int64_t t, int64_t d, gemm_epi_dtype dtype, const void* X,
                                      const void* residual, const void* gamma, float eps,
                                      void* H, void* Q, gemm_epi_scale_mode mode, float* scale,
                                      float* rstd, void* workspace, cudaStream_t stream)
{
    if (mode != GEMM_EPI_SCALE_ROW && mode != GEMM_EPI_SCALE_TENSOR && mode != GEMM_EPI_SCALE_GIVEN)
        return GEMM_EPI_ERR_INVALID_ARG;
    return rmsnorm(t, d, dtype, X, residual, gamma, eps, H, Q, static_cast<int>(mode), scale, rstd,
                   workspace, stream);
}

gemm_epi_status gemm_epi_rmsnorm_backward(int64_t t, int64_t d, gemm_epi_dtype dtype,
                                          const void* dY, const void* H, const void* gamma,
                                          const float* rstd, const void* dH, void* dX,
                                          float* dgamma, void* workspace, cudaStream_t stream)
{
    if (!is_16bit(dtype)) return GEMM_EPI_ERR_INVALID_ARG;
    if (!norm_shape_ok(t, d)) return GEMM_EPI_ERR_UNSUPPORTED_SHAPE;
    if (!dgamma) return GEMM_EPI_ERR_INVALID_ARG;
    if (!aligned(dgamma, 4)) return GEMM_EPI_ERR_MISALIGNED;
    if (t > 0) {
        if (!dY || !H || !gamma || !rstd || !dX || !workspace || dX == H)
            return GEMM_EPI_ERR_INVALID_ARG;
        if (!aligned(dY, 16) || !aligned(H, 16) || !aligned(gamma, 16) || !aligned(rstd, 4) ||
            !aligned(dH, 16) || !aligned(dX, 16) || !aligned(workspace, 16))
            return GEMM_EPI_ERR_MISALIGNED;
        const Buffer y = {dY, 2 * t * d}, h = {H, 2 * t * d}, g = {gamma, 2 * d}, rs = {rstd, 4 * t}, z = {dH, 2 * t * d};
        const Buffer dx = {dX, 2 * t * d}, dg = {dgamma, 4 * d}, ws = {workspace, gemm_epi_rmsnorm_workspace(t, d)};
        if (!apart(dx, {h, g, rs, dg, ws}, {y, z}) || !apart(dg, {y, h, g, rs, z, ws}) || !apart(ws, {y, h, g, rs, z}))
            return GEMM_EPI_ERR_INVALID_ARG;
    }
    int sms = 0;
    const gemm_epi_status st = device_sms(&sms);
    if (st != GEMM_EPI_OK) return st;
    if (t == 0) return launched(cudaMemsetAsync(dgamma, 0, sizeof(float) * static_cast<size_t>(d), stream));
    RmsnormBackwardArgs a;
    a.dY = dY;
    a.H = H;
    a.gamma = gamma;
    a.rstd = rstd;
    a.dH = dH;
    a.dX = dX;
    a.dgamma = dgamma;
    a.ws_mean = static_cast<float*>(workspace);
    a.ws_dgamma = a.ws_mean + round16(sizeof(float) * t) / sizeof(float);
    a.t = static_cast<int>(t);
    a.d = static_cast<int>(d);
    return launched(rmsnorm_backward_launch(a, dtype == GEMM_EPI_BF16, stream));
}

int64_t gemm_epi_rmsnorm_workspace(int64_t t, int64_t d)
{
    if (!norm_shape_ok(t, d)) return 0;
    const int64_t forward = round16(sizeof(uint32_t) * kRmsMaxParts) + round16(sizeof(float) * t);
    const int64_t backward = round16(sizeof(float) * t) + round16(sizeof(float) * rmsnorm_backward_parts(t, d) * d);
    return forward > backward ? forward : backward;
}

gemm_epi_status gemm_epi_w4_matmul(int64_t m, int64_t n, int64_t k, int64_t group,
                                   gemm_epi_dtype dtype, gemm_epi_epilog epilog, const void* A,
                                   const void* W, const void* scales, const uint8_t* zeros,
                                   const void* bias, const void* residual, void* D,
                                   cudaStream_t stream)
{
    if (epilog != GEMM_EPI_BIAS && epilog != GEMM_EPI_RELU_BIAS && epilog != GEMM_EPI_GELU_BIAS &&
        epilog != GEMM_EPI_TANH_BIAS && epilog != GEMM_EPI_BIAS_RESIDUAL && epilog != GEMM_EPI_NONE)
        return GEMM_EPI_ERR_INVALID_ARG;
    gemm_epi_status st = w4_checked(n, k, group, dtype);
    if (st != GEMM_EPI_OK) return st;
    if (m < 0 || m > kW4MaxM) return GEMM_EPI_ERR_UNSUPPORTED_SHAPE;
    if (m == 0 || n == 0) return GEMM_EPI_OK;
    if (!D || (bias != nullptr) != (epilog != GEMM_EPI_NONE) ||
        (residual != nullptr) != (epilog == GEMM_EPI_BIAS_RESIDUAL))
        return GEMM_EPI_ERR_INVALID_ARG;
    if (k > 0 && (!A || !W || !scales)) return GEMM_EPI_ERR_INVALID_ARG;
    if (!aligned(A, 16) || !aligned(W, 16) || !aligned(scales, 16) || !aligned(zeros, 8) ||
        !aligned(bias, 2) || !aligned(residual, 16) || !aligned(D, 16))
        return GEMM_EPI_ERR_MISALIGNED;
    // (blocks write columns of D while others still read all of A)
    const int64_t scaled = k / group * n;
    if (!apart({D, 2 * m * n}, {{A, 2 * m * k}, {W, n * k / 2}, {scales, 2 * scaled}, {zeros, scaled}, {bias, 2 * n}},
               {{residual, 2 * m * n}}))
        return GEMM_EPI_ERR_INVALID_ARG;
    int sms = 0;
    st = device_sms(&sms);
    if (st != GEMM_EPI_OK) return st;
    W4Args a = {};
    a.A = A;
    a.W = W;
    a.scales = scales;
    a.zeros = zeros;
    a.bias = bias;
    a.residual = residual;
    a.D = D;
    a.m = static_cast<int>(m);
    a.n = static_cast<int>(n);
    a.k = static_cast<int>(k);
    a.group = static_cast<int>(group);
    a.epilog = static_cast<int>(epilog);
    return launched(w4_matmul_launch(a, dtype == GEMM_EPI_BF16, sms, stream));
}

gemm_epi_status gemm_epi_w4_dequantize(int64_t n, int64_t k, int64_t group,
                                       gemm_epi_dtype dtype, const void* W, const void* scales,
                                       const uint8_t* zeros, void* B, cudaStream_t stream)
{
    gemm_epi_status st = w4_checked(n, k, group, dtype);
    if (st != GEMM_EPI_OK) return st;
    if (n == 0 || k == 0) return GEMM_EPI_OK;
    if (!W || !scales || !B) return GEMM_EPI_ERR_INVALID_ARG;
    if (!aligned(W, 16) || !aligned(scales, 16) || !aligned(zeros, 8) || !aligned(B, 16))
        return GEMM_EPI_ERR_MISALIGNED;
    const int64_t scaled = k / group * n;
    if (!apart({B, 2 * n * k}, {{W, n * k / 2}, {scales, 2 * scaled}, {zeros, scaled}})) return GEMM_EPI_ERR_INVALID_ARG;
    int sms = 0;
    st = device_sms(&sms);
    if (st != GEMM_EPI_OK) return st;
    W4Args a = {};
    a.W = W;
    a.scales = scales;
    a.zeros = zeros;
    a.D = B;
    a.n = static_cast<int>(n);
    a.k = static_cast<int>(k);
    a.group = static_cast<int>(group);
    return launched(w4_dequantize_launch(a, dtype == GEMM_EPI_BF16, sms, stream));
}

gemm_epi_status gemm_epi_dropout(int64_t count, gemm_epi_dtype dtype, const void* X,
                                 const void* residual, float p, uint64_t seed, uint64_t offset,
                                 const uint64_t* offset_device, void* Y, cudaStream_t stream)
{
    if (!is_16bit(dtype)) return GEMM_EPI_ERR_INVALID_ARG;
    if (count < 0 || count > (1ll << 40)) return GEMM_EPI_ERR_UNSUPPORTED_SHAPE;
    if (!(p >= 0.0f) || !(p <= 1.0f)) return GEMM_EPI_ERR_INVALID_ARG;
    if (count == 0) return GEMM_EPI_OK;
    if (!X || !Y) return GEMM_EPI_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(residual, 16) || !aligned(Y, 16) || !aligned(offset_device, 8))
        return GEMM_EPI_ERR_MISALIGNED;
    if (!apart({Y, 2 * count}, {{offset_device, 8}}, {{X, 2 * count}, {residual, 2 * count}})) return GEMM_EPI_ERR_INVALID_ARG;
    int sms = 0;
    const gemm_epi_status st = device_sms(&sms);
    if (st != GEMM_EPI_OK) return st;
    DropoutArgs a;
    a.X = X;
    a.residual = residual;
    a.Y = Y;
    a.offset_device = reinterpret_cast<const unsigned long long*>(offset_device);
    a.offset = offset;
    a.count = count;
    a.key0 = static_cast<uint32_t>(seed);
    a.key1 = static_cast<uint32_t>(seed >> 32);
    a.drop = static_cast<uint32_t>(std::nearbyint(static_cast<double>(p) * 65536.0));
    a.scale = a.drop == 65536 ? 0.0f : static_cast<float>(65536.0 / (65536.0 - a.drop));
    return launched(dropout_launch(a, dtype == GEMM_EPI_BF16, stream));
}

}  // extern "C"
