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

// Sums over each group's lanes, all rows at once: the shuffles of one row hide
// the latency of another's.
template <int N>
__device__ __forceinline__ void team_sums(float (&v)[N], int lanes)
{
    for (int d = 1; d < lanes; d <<= 1)
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
}

__device__ __forceinline__ float oct_sum(const float2 (&f)[4])
{
    const float2 t = __fadd2_rn(__fadd2_rn(f[0], f[1]), __fadd2_rn(f[2], f[3]));
    return t.x + t.y;
}

template <int DT, bool HOLD>
__global__ void __launch_bounds__(kTokenThreads, DT == TSX_F32 ? 2 : 3)
    norm_token_kernel(NormArgs a, const void* x, const void* weight, const void* bias, void* y, float* mean,
                      float* rstd, HeldOut held)
{
    const NormPlace s = norm_place<true>(a);
    const int lanes = a.per_group / 8;   // threads to a group
    const float m = static_cast<float>(a.per_group), inv_m = 1.f / m;   // a power of two
    Chan<true> k;
    k.params<DT, true>(a, s, weight, bias);
    const int group = s.group0 + local_group(a, s.at.ch);
    const bool first = s.at.ch % a.per_group == 0;
    const int P = a.lay.P;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (P * kTokenRows);
    Oct<DT> o[kTokenRows];
    int64_t base = static_cast<int64_t>(blockIdx.x) * (P * kTokenRows);
    auto load = [&](int64_t from, Oct<DT> (&to)[kTokenRows]) {
#pragma unroll
        for (int i = 0; i < kTokenRows; ++i) {
            const int64_t row = from + i * P + s.p;
            if (s.live && row < a.n)
                to[i] = oct_load<DT, true>(x, row * a.x_pitch + s.ch0, s.at);
            else
                oct_zero(to[i]);
        }
    };
    load(base, o);
    for (; base < a.n; base += stride) {
        Oct<DT> next[kTokenRows];
        load(base + stride, next);
        float mu[kTokenRows], dev[kTokenRows];
#pragma unroll
        for (int i = 0; i < kTokenRows; ++i) {
            float2 f[4];
            oct_floats(o[i], f);
            mu[i] = oct_sum(f);
        }
        team_sums(mu, lanes);
#pragma unroll
        for (int i = 0; i < kTokenRows; ++i) {
            float2 f[4], sq = make_float2(0.f, 0.f);
            oct_floats(o[i], f);
            mu[i] *= inv_m;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 d = __fadd2_rn(f[j], pair_of(-mu[i]));
                sq = __ffma2_rn(d, d, sq);
            }
            dev[i] = sq.x + sq.y;
        }
        team_sums(dev, lanes);
#pragma unroll
        for (int i = 0; i < kTokenRows; ++i) {
            const int64_t row = base + i * P + s.p;
            const bool live = s.live && row < a.n;
            const float rs = rstd_of(dev[i], m, a.eps);
            float2 f[4], out[4];
            oct_floats(o[i], f);
            k.statistics(mu[i], rs);
            k.apply(a, f, out);
            if (live) {
                oct_store<DT, true>(y, row * a.y_pitch + s.ch0, s.at, oct_round<DT>(out));
                if (first) {
                    mean[row * a.groups + group] = mu[i];
                    rstd[row * a.groups + group] = rs;
                }
            }
            if constexpr (HOLD)
                hold<true>(a, s, f, live, row, held);
            o[i] = next[i];
        }
    }
}

template <int DT, bool HELD>
__global__ void __launch_bounds__(kTokenThreads, 2)
    norm_token_grad_kernel(NormArgs a, const void* dy, Saved x, const void* weight, const void* bias,
                           const float* mean, const float* rstd, void* dx, float* chan)
{
    extern __shared__ float2 shared[];
    const NormPlace s = norm_place<true>(a);
    const int lanes = a.per_group / 8;
    const float minus_m = -1.f / static_cast<float>(a.per_group);
    Chan<true> k;
    k.params<DT, true>(a, s, weight, bias);
    const int group = s.group0 + local_group(a, s.at.ch);
    const int P = a.lay.P;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (P * kTokenGradRows);
    struct Row {
        GradRow<DT, true, HELD> g;
        float mu, rs;
    };
    Row cur[kTokenGradRows];
    auto load = [&](int64_t from, Row (&to)[kTokenGradRows]) {
#pragma unroll
        for (int i = 0; i < kTokenGradRows; ++i) {
            const int64_t row = from + i * P + s.p;
            if (s.live && row < a.n) {
                to[i].g.load(a, s, dy, x, row);
                to[i].mu = __ldg(mean + row * a.groups + group);
                to[i].rs = __ldg(rstd + row * a.groups + group);
            }
        }
    };
    float2 sz[4], szx[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        sz[j] = szx[j] = make_float2(0.f, 0.f);
    int64_t base = static_cast<int64_t>(blockIdx.x) * (P * kTokenGradRows);
    load(base, cur);
    for (; base < a.n; base += stride) {
        Row next[kTokenGradRows];
        load(base + stride, next);
        float2 hat[kTokenGradRows][4], dz[kTokenGradRows][4];
        float s1[kTokenGradRows], s2[kTokenGradRows];
#pragma unroll
        for (int i = 0; i < kTokenGradRows; ++i) {
            s1[i] = s2[i] = 0.f;
            if (s.live && base + i * P + s.p < a.n) {
                float2 fd[4], fx[4], t1 = make_float2(0.f, 0.f), t2 = t1;
                oct_floats(cur[i].g.dy, fd);
                cur[i].g.saved_floats(a, fx);
                k.statistics(cur[i].mu, cur[i].rs);
                k.slopes(a, fd, fx, hat[i], dz[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 dzx = __fmul2_rn(dz[i][j], hat[i][j]);
                    sz[j] = __fadd2_rn(sz[j], dz[i][j]);
                    szx[j] = __fadd2_rn(szx[j], dzx);
                    t1 = __ffma2_rn(dz[i][j], k.w[j], t1);
                    t2 = __ffma2_rn(dzx, k.w[j], t2);
                }
                s1[i] = t1.x + t1.y;
                s2[i] = t2.x + t2.y;
            }
        }
        team_sums(s1, lanes);
        team_sums(s2, lanes);
#pragma unroll
        for (int i = 0; i < kTokenGradRows; ++i) {
            const int64_t row = base + i * P + s.p;
            if (s.live && row < a.n) {
                Grouped<true> g1, g2;
                g1.v[0] = pair_of(s1[i] * minus_m);
                g2.v[0] = pair_of(s2[i] * minus_m);
                float2 out[4];
                k.statistics(cur[i].mu, cur[i].rs);
                k.gradient(dz[i], hat[i], g1, g2, out);
                oct_store<DT, true>(dx, row * a.x_pitch + s.ch0, s.at, oct_round<DT>(out));
            }
            cur[i] = next[i];
        }
    }
    const int width = s.at.cols, slot = slot_stride(width);
    float2* work = shared;                      // [threads]
    float2* columns = work + kTokenThreads;     // [run_cols]
    float2* slots = columns + a.lay.run_cols;   // [P][stride]
    if (s.live)
        leave_sums(s.at, sz, szx, slots + s.p * slot);
    __syncthreads();
    sum_lanes(slots, slot, 1, P, width, columns, work);
    float* out = chan + static_cast<int64_t>(blockIdx.x) * 2 * a.c + s.ch0;
    for (int ch = threadIdx.x; ch < width; ch += blockDim.x) {
        out[ch] = columns[ch].y;
        out[a.c + ch] = columns[ch].x;
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
    const size_t slots =
        (kTokenThreads + a.lay.run_cols + size_t(a.lay.P) * slot_stride(a.lay.run_cols)) * sizeof(float2);
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
