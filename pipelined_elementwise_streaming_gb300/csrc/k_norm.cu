// Group norm over samples too long to be held on chip, or of any layout: the
// streaming kernels, which read their operands twice.  The first kernel sums
// over ranges of rows (one CTA to a range of a run of channels), the second
// joins the ranges' sums and applies.  HBM bounds the first; the second reads
// out of L2 what of the tensor still is there.

#include "tsx_norm.cuh"

namespace tsx {
namespace {

using namespace dev;

constexpr int kRowsAtOnce = 4;   // rows whose loads a thread issues before it uses the first

// A CTA's range of rows: blockIdx.x counts ranges sample by sample.
struct Range {
    int64_t sample, split;
    int64_t row0;   // first row, counted through all samples
    int rows;       // rows of the range
};

__device__ __forceinline__ Range range_of(const NormArgs& a)
{
    Range r;
    const unsigned splits = static_cast<unsigned>(a.lay.splits);
    r.sample = blockIdx.x / splits;
    r.split = blockIdx.x % splits;
    r.row0 = r.sample * a.l + r.split * a.lay.range;
    r.rows = static_cast<int>(min(a.lay.range, a.l - r.split * a.lay.range));
    return r;
}

// A range's place among the parts of its sample.
__device__ __forceinline__ float2* part_of(const NormArgs& a, const NormPlace& s, const Range& r, float2* part)
{
    return part + ((r.sample * a.lay.splits + r.split) * a.lay.pieces + s.piece) * a.groups + s.group0;
}

// ------------------------------------------------------------- forward

// First kernel: (mean, M2) of every range, run and group.
template <int DT, bool VEC, bool BY_OCT>
__global__ void __launch_bounds__(kLayerThreads) norm_stats_kernel(NormArgs a, const void* x, float2* part)
{
    extern __shared__ float2 slots[];   // [P][width], then P counts
    const NormPlace s = norm_place<VEC>(a);
    const Range r = range_of(a);
    const int P = a.lay.P;
    Triples<BY_OCT ? 1 : 8> t;
    t.clear();
    for (int r0 = s.p; s.live && r0 < r.rows; r0 += kRowsAtOnce * P) {
        Oct<DT> o[kRowsAtOnce];
        int have = 0;
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i)
            if (r0 + i * P < r.rows) {
                o[i] = oct_load<DT, VEC>(x, (r.row0 + r0 + i * P) * a.x_pitch + s.ch0, s.at);
                have = i + 1;
            }
        float f[kRowsAtOnce][8];
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i)
            oct_floats(o[i], f[i]);
        t.add_rows(f, have);
    }
    const int width = run_width<BY_OCT>(s);
    float* counts = reinterpret_cast<float*>(slots + P * width);
    join_lanes(s, s.p, P, slots, counts, width, t);
    if (s.live && s.p == 0) {
        if constexpr (BY_OCT) {
            slots[s.at.ch / 8] = make_float2(t.mean[0], t.m2[0]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (s.at.ch + j * s.at.step < s.at.cols)
                    slots[s.at.ch + j * s.at.step] = make_float2(t.mean[j], t.m2[j]);
        }
    }
    __syncthreads();
    join_columns(slots, s.groups, group_cols(a, s) / (BY_OCT ? 8 : 1), r.rows * (BY_OCT ? 8.f : 1.f),
                 part_of(a, s, r, part));
}

// The statistics of the run's groups from their parts, into `stats` [groups]
// as (mean, rstd).  Neighbouring threads read neighbouring groups.  Ends with
// the CTA synchronised.
__device__ __forceinline__ void join_parts(const NormArgs& a, const NormPlace& s, int64_t sample, const float2* part,
                                           float2* stats, float4* work)
{
    const int count = static_cast<int>(a.lay.splits) * a.lay.pieces;
    const float2* first = part + sample * count * a.groups + s.group0;
    const float m = static_cast<float>(a.l) * static_cast<float>(a.per_group);
    const int threads = static_cast<int>(blockDim.x);
    // `lanes` threads to a group, each joins every lanes-th part
    const int lanes = s.groups < threads ? threads / s.groups : 1;
    for (int i = threadIdx.x; i < lanes * s.groups; i += threads) {
        const int lane = i / s.groups, g = i - lane * s.groups;
        Triples<1> t;
        t.clear();
        int split = lane / a.lay.pieces, piece = lane - split * a.lay.pieces;
#pragma unroll 4
        for (int k = lane; k < count; k += lanes) {
            const float2 v = first[static_cast<int64_t>(k) * a.groups + g];
            if (a.lay.pieces == 1) {
                split = k;
            } else {
                split = k / a.lay.pieces;
                piece = k - split * a.lay.pieces;
            }
            const float rows = static_cast<float>(min(a.lay.range, a.l - split * a.lay.range));
            const int cols =
                a.lay.pieces == 1 ? a.per_group : min(a.lay.run_cols, a.per_group - piece * a.lay.run_cols);
            const float mu[1] = {v.x}, dev[1] = {v.y};
            t.join(rows * static_cast<float>(cols), mu, dev);
        }
        work[i] = make_float4(t.count, t.mean[0], t.m2[0], 0.f);
    }
    __syncthreads();
    for (int g = threadIdx.x; g < s.groups; g += threads) {
        Triples<1> t;
        t.clear();
        for (int k = 0; k < lanes; ++k) {
            const float4 v = work[k * s.groups + g];
            const float mu[1] = {v.y}, dev[1] = {v.z};
            t.join(v.x, mu, dev);
        }
        stats[g] = make_float2(t.mean[0], rstd_of(t.m2[0], m, a.eps));
    }
    __syncthreads();
}

// Second kernel: y, and with HOLD the checkpoint of x.
template <int DT, bool VEC, bool BY_OCT, bool HOLD>
__global__ void __launch_bounds__(kLayerThreads)
    norm_apply_kernel(NormArgs a, const void* x, const void* weight, const void* bias, void* y, float* mean,
                      float* rstd, HeldOut held, const float2* part)
{
    extern __shared__ float4 work[];   // [threads or groups], then [run_groups] statistics
    const NormPlace s = norm_place<VEC>(a);
    const Range r = range_of(a);
    Chan<BY_OCT> k;
    k.template params<DT, VEC>(a, s, weight, bias);
    float2* stats = reinterpret_cast<float2*>(work + max(static_cast<int>(blockDim.x), a.lay.run_groups));
    join_parts(a, s, r.sample, part, stats, work);
    k.statistics(a, s, stats);
    if (r.split == 0 && s.piece == 0)
        for (int g = threadIdx.x; g < s.groups; g += blockDim.x) {
            mean[r.sample * a.groups + s.group0 + g] = stats[g].x;
            rstd[r.sample * a.groups + s.group0 + g] = stats[g].y;
        }
    const int P = a.lay.P;
    // whole warps walk together: the teams' shuffles need every lane
    for (int base = 0; base < r.rows; base += kRowsAtOnce * P) {
        const int r0 = base + s.p;
        Oct<DT> o[kRowsAtOnce];
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i)
            if (s.live && r0 + i * P < r.rows)
                o[i] = oct_load<DT, VEC>(x, (r.row0 + r0 + i * P) * a.x_pitch + s.ch0, s.at);
            else
                oct_zero(o[i]);
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i) {
            const int64_t row = r.row0 + r0 + i * P;
            const bool live = s.live && r0 + i * P < r.rows;
            float f[8], out[8];
            oct_floats(o[i], f);
            k.template apply<DT>(a, f, out);
            if (live)
                oct_store<DT, VEC>(y, row * a.y_pitch + s.ch0, s.at, oct_round<DT>(out));
            if constexpr (HOLD)
                hold<VEC>(a, s, f, live, row, held);
        }
    }
}

// ------------------------------------------------------------ backward

__device__ __forceinline__ void load_stats(const NormArgs& a, const NormPlace& s, int64_t sample, const float* mean,
                                           const float* rstd, float2* stats)
{
    for (int g = threadIdx.x; g < s.groups; g += blockDim.x) {
        const int64_t at = sample * a.groups + s.group0 + g;
        stats[g] = make_float2(mean[at], rstd[at]);
    }
    __syncthreads();
}

constexpr int kGradRows = 2;   // two operands: half as many rows at once

// First kernel: S1 and S2 of every range, run and group, and the range's sums
// for dweight and dbias.
template <int DT, bool VEC, bool BY_OCT, bool HELD>
__global__ void __launch_bounds__(kLayerThreads)
    norm_sums_kernel(NormArgs a, const void* dy, Saved x, const void* weight, const void* bias, const float* mean,
                     const float* rstd, float2* part, float* chan)
{
    extern __shared__ float2 shared[];
    const NormPlace s = norm_place<VEC>(a);
    const Range r = range_of(a);
    float2* stats = shared;                       // [run_groups]
    float2* slots = shared + a.lay.run_groups;    // [P][run_cols]
    Chan<BY_OCT> k;
    k.template params<DT, VEC>(a, s, weight, bias);
    load_stats(a, s, r.sample, mean, rstd, stats);
    k.statistics(a, s, stats);
    float sz[8], szx[8];   // sums of dz and dz xhat, channel by channel
#pragma unroll
    for (int j = 0; j < 8; ++j)
        sz[j] = szx[j] = 0.f;
    const int P = a.lay.P;
    for (int r0 = s.p; s.live && r0 < r.rows; r0 += kGradRows * P) {
        GradRow<DT, VEC, HELD> g[kGradRows];
#pragma unroll
        for (int i = 0; i < kGradRows; ++i)
            if (r0 + i * P < r.rows)
                g[i].load(a, s, dy, x, r.row0 + r0 + i * P);
#pragma unroll
        for (int i = 0; i < kGradRows; ++i)
            if (r0 + i * P < r.rows) {
                float fd[8], fx[8], hat[8], dz[8];
                g[i].floats(a, fd, fx);
                k.template slopes<DT>(a, fd, fx, hat, dz);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sz[j] += dz[j];
                    szx[j] += dz[j] * hat[j];
                }
            }
    }
    add_lanes(s, s.p, P, slots, s.at.cols, sz, szx);
    if (s.live && s.p == 0) {
        float* out = chan + (r.sample * a.lay.splits + r.split) * 2 * a.c + s.ch0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int ch = s.at.ch + j * s.at.step;
            if (ch < s.at.cols) {
                slots[ch] = make_float2(sz[j], szx[j]);
                out[ch] = szx[j];
                out[a.c + ch] = sz[j];
            }
        }
    }
    __syncthreads();
    weigh_columns<DT>(a, s, weight, slots, part_of(a, s, r, part));
}

// Second kernel: dx.
template <int DT, bool VEC, bool BY_OCT, bool HELD>
__global__ void __launch_bounds__(kLayerThreads)
    norm_grad_kernel(NormArgs a, const void* dy, Saved x, const void* weight, const void* bias, const float* mean,
                     const float* rstd, void* dx, const float2* part)
{
    extern __shared__ float2 shared[];
    const NormPlace s = norm_place<VEC>(a);
    const Range r = range_of(a);
    float2* stats = shared;                      // [run_groups]
    float2* sums = stats + a.lay.run_groups;     // [run_groups]: S1 / M, S2 / M
    float2* work = sums + a.lay.run_groups;      // [threads or groups]
    Chan<BY_OCT> k;
    k.template params<DT, VEC>(a, s, weight, bias);
    const int count = static_cast<int>(a.lay.splits) * a.lay.pieces;
    const float2* first = part + r.sample * count * a.groups + s.group0;
    const float m = static_cast<float>(a.l) * static_cast<float>(a.per_group);
    const int threads = static_cast<int>(blockDim.x);
    const int lanes = s.groups < threads ? threads / s.groups : 1;
    for (int i = threadIdx.x; i < lanes * s.groups; i += threads) {
        const int lane = i / s.groups, g = i - lane * s.groups;
        float2 t = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int n = lane; n < count; n += lanes) {
            const float2 v = first[static_cast<int64_t>(n) * a.groups + g];
            t.x += v.x;
            t.y += v.y;
        }
        work[i] = t;
    }
    __syncthreads();
    for (int g = threadIdx.x; g < s.groups; g += threads) {
        float2 t = work[g];
        for (int n = 1; n < lanes; ++n) {
            t.x += work[n * s.groups + g].x;
            t.y += work[n * s.groups + g].y;
        }
        sums[g] = make_float2(t.x / m, t.y / m);
    }
    load_stats(a, s, r.sample, mean, rstd, stats);   // synchronises
    k.statistics(a, s, stats);
    float s1[BY_OCT ? 1 : 8], s2[BY_OCT ? 1 : 8];
#pragma unroll
    for (int j = 0; j < (BY_OCT ? 1 : 8); ++j) {
        const int ch = s.at.ch + j * s.at.step;
        const float2 t = sums[ch < s.at.cols ? local_group(a, ch) : 0];
        s1[j] = t.x;
        s2[j] = t.y;
    }
    const int P = a.lay.P;
    for (int r0 = s.p; s.live && r0 < r.rows; r0 += kGradRows * P) {
        GradRow<DT, VEC, HELD> g[kGradRows];
#pragma unroll
        for (int i = 0; i < kGradRows; ++i)
            if (r0 + i * P < r.rows)
                g[i].load(a, s, dy, x, r.row0 + r0 + i * P);
#pragma unroll
        for (int i = 0; i < kGradRows; ++i)
            if (r0 + i * P < r.rows) {
                float fd[8], fx[8], hat[8], dz[8], out[8];
                g[i].floats(a, fd, fx);
                k.template slopes<DT>(a, fd, fx, hat, dz);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    out[j] = k.rs(j) * (dz[j] * k.w[j] - s1[BY_OCT ? 0 : j] - hat[j] * s2[BY_OCT ? 0 : j]);
                oct_store<DT, VEC>(dx, (r.row0 + r0 + i * P) * a.x_pitch + s.ch0, s.at, oct_round<DT>(out));
            }
    }
}

// dweight and dbias: the sums of the [slices][2][c] partial sums, slice after
// slice within each of 32 lanes, then the lanes by halves.
constexpr int kParamCols = 32, kParamLanes = 32;
__global__ void __launch_bounds__(kParamCols* kParamLanes)
    norm_params_kernel(const float* chan, int64_t slices, int c, float* dweight, float* dbias)
{
    __shared__ float part[kParamLanes][kParamCols];
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kParamCols + threadIdx.x;   // of 2 c
    float t = 0.f;
    if (col < 2 * static_cast<int64_t>(c)) {
#pragma unroll 8
        for (int64_t i = threadIdx.y; i < slices; i += kParamLanes)
            t += chan[i * 2 * c + col];
    }
    part[threadIdx.y][threadIdx.x] = t;
    for (int half = kParamLanes / 2; half > 0; half >>= 1) {
        __syncthreads();
        if (static_cast<int>(threadIdx.y) < half)
            part[threadIdx.y][threadIdx.x] += part[threadIdx.y + half][threadIdx.x];
    }
    if (threadIdx.y == 0 && col < 2 * static_cast<int64_t>(c)) {
        if (col < c)
            dweight[col] = part[0][threadIdx.x];
        else
            dbias[col - c] = part[0][threadIdx.x];
    }
}

__global__ void norm_empty_kernel(float* mean, float* rstd, int64_t count, float eps)
{
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < count;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        mean[i] = 0.f;
        rstd[i] = 1.f / sqrtf(eps);
    }
}

}  // namespace

cudaError_t launch_norm(int dtype, const NormArgs& a, const void* x, const void* weight, const void* bias, void* y,
                        float* mean, float* rstd, HeldOut held, NormScratch scratch, cudaStream_t st)
{
    const NormLayout& lay = a.lay;
    const dim3 grid(unsigned(a.n * lay.splits), unsigned(lay.runs));
    const int width = lay.oct_in_group ? lay.run_cols / 8 : lay.run_cols;
    const size_t slots = size_t(lay.P) * width * sizeof(float2) + lay.P * sizeof(float);
    const int items = lay.threads > lay.run_groups ? lay.threads : lay.run_groups;
    const size_t stats = items * sizeof(float4) + lay.run_groups * sizeof(float2);
#define CALL(DT, VEC, BY_OCT) \
    norm_stats_kernel<DT, VEC, BY_OCT><<<grid, lay.threads, slots, st>>>(a, x, scratch.part)
    TSX_BY_LAYOUT(dtype, lay, CALL);
#undef CALL
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
#define CALL(DT, VEC, BY_OCT)                                                                                \
    if (held.q)                                                                                              \
        norm_apply_kernel<DT, VEC, BY_OCT, true>                                                             \
            <<<grid, lay.threads, stats, st>>>(a, x, weight, bias, y, mean, rstd, held, scratch.part);       \
    else                                                                                                     \
        norm_apply_kernel<DT, VEC, BY_OCT, false>                                                            \
            <<<grid, lay.threads, stats, st>>>(a, x, weight, bias, y, mean, rstd, held, scratch.part)
    TSX_BY_LAYOUT(dtype, lay, CALL);
#undef CALL
    return cudaGetLastError();
}

cudaError_t launch_norm_backward(int dtype, const NormArgs& a, const void* dy, Saved x, const void* weight,
                                 const void* bias, const float* mean, const float* rstd, void* dx, float* dweight,
                                 float* dbias, NormScratch scratch, cudaStream_t st)
{
    const NormLayout& lay = a.lay;
    const dim3 grid(unsigned(a.n * lay.splits), unsigned(lay.runs));
    const size_t sums = (size_t(lay.run_groups) + size_t(lay.P) * lay.run_cols) * sizeof(float2);
#define CALL(DT, VEC, BY_OCT)                                                                                    \
    if (x.q)                                                                                                     \
        norm_sums_kernel<DT, VEC, BY_OCT, true><<<grid, lay.threads, sums, st>>>(a, dy, x, weight, bias, mean,    \
                                                                                 rstd, scratch.part, scratch.chan); \
    else                                                                                                         \
        norm_sums_kernel<DT, VEC, BY_OCT, false><<<grid, lay.threads, sums, st>>>(a, dy, x, weight, bias, mean,   \
                                                                                  rstd, scratch.part, scratch.chan)
    TSX_BY_LAYOUT(dtype, lay, CALL);
#undef CALL
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    const int items = lay.threads > lay.run_groups ? lay.threads : lay.run_groups;
    const size_t stats = (2 * size_t(lay.run_groups) + items) * sizeof(float2);
#define CALL(DT, VEC, BY_OCT)                                                                               \
    if (x.q)                                                                                                \
        norm_grad_kernel<DT, VEC, BY_OCT, true>                                                             \
            <<<grid, lay.threads, stats, st>>>(a, dy, x, weight, bias, mean, rstd, dx, scratch.part);       \
    else                                                                                                    \
        norm_grad_kernel<DT, VEC, BY_OCT, false>                                                            \
            <<<grid, lay.threads, stats, st>>>(a, dy, x, weight, bias, mean, rstd, dx, scratch.part)
    TSX_BY_LAYOUT(dtype, lay, CALL);
#undef CALL
    e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    return launch_norm_params(a, a.n * lay.splits, scratch.chan, dweight, dbias, st);
}

cudaError_t launch_norm_params(const NormArgs& a, int64_t slices, const float* chan, float* dweight, float* dbias,
                               cudaStream_t st)
{
    const int64_t cols = 2 * int64_t(a.c);
    norm_params_kernel<<<unsigned((cols + kParamCols - 1) / kParamCols), dim3(kParamCols, kParamLanes), 0, st>>>(
        chan, slices, a.c, dweight, dbias);
    return cudaGetLastError();
}

cudaError_t launch_norm_empty(float* mean, float* rstd, int64_t count, float eps, cudaStream_t st)
{
    const int64_t blocks = (count + 255) / 256;
    norm_empty_kernel<<<unsigned(blocks < 1024 ? blocks : 1024), 256, 0, st>>>(mean, rstd, count, eps);
    return cudaGetLastError();
}

}  // namespace tsx
