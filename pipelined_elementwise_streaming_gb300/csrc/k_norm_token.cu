// Group norm of tokens (l = 1) whose groups are a power of two of octs, at
// most a warp's 32: every group lies in neighbouring lanes of one warp, so its
// sums are a few shuffles and a row is read once, with no shared memory and no
// barrier.  HBM bounds it.  A CTA walks rows so that weight and bias (and the
// sums for their gradients) stay in registers.

#include "tsx_norm.cuh"

namespace tsx {
namespace {

using namespace dev;

constexpr int kTokenRows = 4;       // rows whose loads a thread issues before it uses the first
constexpr int kTokenGradRows = 2;   // two operands a row

template <int DT, bool HOLD>
__global__ void __launch_bounds__(kLayerThreads)
    norm_token_kernel(NormArgs a, const void* x, const void* weight, const void* bias, void* y, float* mean,
                      float* rstd, HeldOut held)
{
    const NormPlace s = norm_place<true>(a);
    const int lanes = a.per_group / 8;   // threads to a group
    const float m = static_cast<float>(a.per_group);
    Chan<true> k;
    k.params<DT, true>(a, s, weight, bias);
    const bool first = s.at.ch % a.per_group == 0;
    const int group = s.group0 + local_group(a, s.at.ch);
    const int P = a.lay.P;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * (P * kTokenRows); base < a.n;
         base += static_cast<int64_t>(gridDim.x) * (P * kTokenRows)) {
        Oct<DT> o[kTokenRows];
#pragma unroll
        for (int i = 0; i < kTokenRows; ++i) {
            const int64_t row = base + i * P + s.p;
            if (s.live && row < a.n)
                o[i] = oct_load<DT, true>(x, row * a.x_pitch + s.ch0, s.at);
            else
                oct_zero(o[i]);
        }
#pragma unroll
        for (int i = 0; i < kTokenRows; ++i) {
            const int64_t row = base + i * P + s.p;
            const bool live = s.live && row < a.n;
            float f[8], out[8], sum = 0.f, dev = 0.f;
            oct_floats(o[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                sum += f[j];
            k.mean[0] = lanes_sum(sum, lanes) / m;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = f[j] - k.mean[0];
                dev += d * d;
            }
            k.rstd[0] = rstd_of(lanes_sum(dev, lanes), m, a.eps);
            k.apply<DT>(a, f, out);
            if (live) {
                oct_store<DT, true>(y, row * a.y_pitch + s.ch0, s.at, oct_round<DT>(out));
                if (first) {
                    mean[row * a.groups + group] = k.mean[0];
                    rstd[row * a.groups + group] = k.rstd[0];
                }
            }
            if constexpr (HOLD)
                hold<true>(a, s, f, live, row, held);
        }
    }
}

template <int DT, bool HELD>
__global__ void __launch_bounds__(kLayerThreads)
    norm_token_grad_kernel(NormArgs a, const void* dy, Saved x, const void* weight, const void* bias,
                           const float* mean, const float* rstd, void* dx, float* chan)
{
    extern __shared__ float2 slots[];   // [P][run_cols]
    const NormPlace s = norm_place<true>(a);
    const int lanes = a.per_group / 8;
    const float inv_m = 1.f / static_cast<float>(a.per_group);
    Chan<true> k;
    k.params<DT, true>(a, s, weight, bias);
    const int group = s.group0 + local_group(a, s.at.ch);
    const int P = a.lay.P;
    float sz[8], szx[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        sz[j] = szx[j] = 0.f;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * (P * kTokenGradRows); base < a.n;
         base += static_cast<int64_t>(gridDim.x) * (P * kTokenGradRows)) {
        GradRow<DT, true, HELD> g[kTokenGradRows];
        float mu[kTokenGradRows], rs[kTokenGradRows];
#pragma unroll
        for (int i = 0; i < kTokenGradRows; ++i) {
            const int64_t row = base + i * P + s.p;
            mu[i] = rs[i] = 0.f;
            if (s.live && row < a.n) {
                g[i].load(a, s, dy, x, row);
                mu[i] = __ldg(mean + row * a.groups + group);
                rs[i] = __ldg(rstd + row * a.groups + group);
            }
        }
#pragma unroll
        for (int i = 0; i < kTokenGradRows; ++i) {
            const int64_t row = base + i * P + s.p;
            const bool live = s.live && row < a.n;
            float fd[8], fx[8], hat[8], dz[8], s1 = 0.f, s2 = 0.f;
            k.mean[0] = mu[i];
            k.rstd[0] = rs[i];
            if (live) {
                g[i].floats(a, fd, fx);
                k.slopes<DT>(a, fd, fx, hat, dz);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sz[j] += dz[j];
                    szx[j] += dz[j] * hat[j];
                    dz[j] *= k.w[j];
                    s1 += dz[j];
                    s2 += dz[j] * hat[j];
                }
            }
            s1 = lanes_sum(s1, lanes) * inv_m;
            s2 = lanes_sum(s2, lanes) * inv_m;
            if (live) {
                float out[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    out[j] = rs[i] * (dz[j] - s1 - hat[j] * s2);
                oct_store<DT, true>(dx, row * a.x_pitch + s.ch0, s.at, oct_round<DT>(out));
            }
        }
    }
    add_lanes(s, s.p, P, slots, s.at.cols, sz, szx);
    if (s.live && s.p == 0) {
        float* out = chan + static_cast<int64_t>(blockIdx.x) * 2 * a.c + s.ch0 + s.at.ch;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            out[j] = szx[j];
            out[a.c + j] = sz[j];
        }
    }
}

}  // namespace

cudaError_t launch_norm_token(int dtype, const NormArgs& a, const void* x, const void* weight, const void* bias,
                              void* y, float* mean, float* rstd, HeldOut held, cudaStream_t st)
{
    const dim3 grid(unsigned(a.lay.splits), unsigned(a.lay.runs));
#define CALL(DT)                                                                                                  \
    if (held.q)                                                                                                   \
        norm_token_kernel<DT, true><<<grid, a.lay.threads, 0, st>>>(a, x, weight, bias, y, mean, rstd, held);     \
    else                                                                                                          \
        norm_token_kernel<DT, false><<<grid, a.lay.threads, 0, st>>>(a, x, weight, bias, y, mean, rstd, held)
    if (dtype == TSX_F16) { CALL(TSX_F16); }
    else if (dtype == TSX_BF16) { CALL(TSX_BF16); }
    else { CALL(TSX_F32); }
#undef CALL
    return cudaGetLastError();
}

cudaError_t launch_norm_token_backward(int dtype, const NormArgs& a, const void* dy, Saved x, const void* weight,
                                       const void* bias, const float* mean, const float* rstd, void* dx,
                                       float* dweight, float* dbias, NormScratch scratch, cudaStream_t st)
{
    const dim3 grid(unsigned(a.lay.splits), unsigned(a.lay.runs));
    const size_t slots = size_t(a.lay.P) * a.lay.run_cols * sizeof(float2);
#define CALL(DT)                                                                                              \
    if (x.q)                                                                                                  \
        norm_token_grad_kernel<DT, true>                                                                      \
            <<<grid, a.lay.threads, slots, st>>>(a, dy, x, weight, bias, mean, rstd, dx, scratch.chan);       \
    else                                                                                                      \
        norm_token_grad_kernel<DT, false>                                                                     \
            <<<grid, a.lay.threads, slots, st>>>(a, dy, x, weight, bias, mean, rstd, dx, scratch.chan)
    if (dtype == TSX_F16) { CALL(TSX_F16); }
    else if (dtype == TSX_BF16) { CALL(TSX_BF16); }
    else { CALL(TSX_F32); }
#undef CALL
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    return launch_norm_params(a, a.lay.splits, scratch.chan, dweight, dbias, st);
}

}  // namespace tsx
