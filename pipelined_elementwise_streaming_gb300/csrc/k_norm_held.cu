// Group norm of samples that fit on chip: a CTA, or a cluster of CTAs that
// share a sample's rows, holds a run of channels of a sample in registers, so
// that its operands are read once.  HBM bounds it, and for small tensors the
// chain load - sum - barrier - store.
//
// A thread holds up to kHeldRows rows of its oct.  The statistics go through
// the CTA's shared memory (tsx_norm.cuh) and, in a cluster, through every
// CTA's copy of the groups' sums: all ranks join the ranks' sums in the same
// order, so they agree to the bit.  A CTA takes Q small samples side by side.

#include "tsx_norm.cuh"

namespace tsx {
namespace {

using namespace dev;

constexpr int kHeldRows = kNormHeldRows;
constexpr int kHeldGradRows = kNormHeldGradRows;

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// A pair in the shared memory of the cluster's CTA `rank`, at the place that
// `p` has in this one.
__device__ __forceinline__ float2 cluster_pair(const float2* p, int rank)
{
    const uint32_t here = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    uint32_t there;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(there) : "memory");
    return v;
}

// Which rows a thread holds: lane, lane + lanes, ... of its sample's part.
struct HeldPlace {
    int rank;         // of the cluster's `ranks` CTAs
    int q, lane;      // sample of the CTA, row lane of the sample
    int64_t tile;     // first sample / samples to a CTA
    int64_t sample;
    int64_t row0;     // the part's first row, counted through all samples
    int rows;         // rows of the part
};

__device__ __forceinline__ HeldPlace held_place(const NormArgs& a, NormPlace& s)
{
    const NormLayout& lay = a.lay;
    HeldPlace h;
    h.tile = blockIdx.x / lay.ranks;
    h.rank = blockIdx.x % lay.ranks;
    h.q = s.p / lay.lanes;
    h.lane = s.p - h.q * lay.lanes;
    h.sample = h.tile * lay.samples + h.q;
    s.live = s.live && h.sample < a.n;
    const int64_t start = h.rank * lay.range;
    h.row0 = h.sample * a.l + start;
    h.rows = static_cast<int>(max(min(lay.range, a.l - start), static_cast<int64_t>(0)));
    return h;
}

// Rows of rank k's part.
__device__ __forceinline__ float rows_of_rank(const NormArgs& a, int k)
{
    return static_cast<float>(max(min(a.lay.range, a.l - k * a.lay.range), static_cast<int64_t>(0)));
}

template <int DT, bool BY_OCT, bool HOLD>
__global__ void __launch_bounds__(kLayerThreads)
    norm_held_kernel(NormArgs a, const void* x, const void* weight, const void* bias, void* y, float* mean,
                     float* rstd, HeldOut held)
{
    extern __shared__ float2 shared[];
    const NormLayout& lay = a.lay;
    NormPlace s = norm_place<true>(a);
    const HeldPlace h = held_place(a, s);
    Oct<DT> o[kHeldRows];
    int have = 0;   // rows that the thread holds
#pragma unroll
    for (int i = 0; i < kHeldRows; ++i) {
        const int r = h.lane + i * lay.lanes;
        oct_zero(o[i]);
        if (s.live && r < h.rows) {
            o[i] = oct_load<DT, true>(x, (h.row0 + r) * a.x_pitch + s.ch0, s.at);
            have = i + 1;
        }
    }
    Chan<BY_OCT> k;
    k.template params<DT, true>(a, s, weight, bias);

    const int width = run_width<BY_OCT>(s), items = lay.samples * s.groups;
    float2* slots = shared;                          // [P][width]
    float2* columns = slots + lay.P * width;         // [samples][width]
    float2* sums = columns + lay.samples * width;    // [samples][groups]: (mean, M2) of the part
    float2* stats = sums + items;                    // [samples][groups]: (mean, rstd)
    float* counts = reinterpret_cast<float*>(stats + items);   // [P]
    Triples<BY_OCT ? 1 : 8> t;
    t.clear();
#pragma unroll
    for (int i0 = 0; i0 < kHeldRows; i0 += 4) {
        float f[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            oct_floats(o[i0 + i], f[i]);
        t.add_rows(f, min(max(have - i0, 0), 4));
    }
    join_lanes(s, h.lane, lay.lanes, slots, counts, width, t);
    if (s.p < lay.P && s.at.ch < s.at.cols && h.lane == 0) {   // absent samples leave zeros
        if constexpr (BY_OCT) {
            columns[h.q * width + s.at.ch / 8] = make_float2(t.mean[0], t.m2[0]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                columns[h.q * width + s.at.ch + j] = make_float2(t.mean[j], t.m2[j]);
        }
    }
    __syncthreads();
    join_columns(columns, items, a.per_group / (BY_OCT ? 8 : 1), h.rows * (BY_OCT ? 8.f : 1.f), sums);
    if (lay.ranks > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    const float m = static_cast<float>(a.l) * static_cast<float>(a.per_group);
    for (int i = threadIdx.x; i < items; i += blockDim.x) {
        float2 v = sums[i];
        if (lay.ranks > 1) {
            Triples<1> j;
            j.clear();
            for (int r = 0; r < lay.ranks; ++r) {
                const float2 u = cluster_pair(&sums[i], r);
                const float mu[1] = {u.x}, dev[1] = {u.y};
                j.join(rows_of_rank(a, r) * a.per_group, mu, dev);
            }
            v = make_float2(j.mean[0], j.m2[0]);
        }
        v.y = rstd_of(v.y, m, a.eps);
        stats[i] = v;
        const int q = i / s.groups;
        const int64_t sample = h.tile * lay.samples + q;
        if (h.rank == 0 && sample < a.n) {
            mean[sample * a.groups + s.group0 + i - q * s.groups] = v.x;
            rstd[sample * a.groups + s.group0 + i - q * s.groups] = v.y;
        }
    }
    if (lay.ranks > 1)
        cluster_arrive();   // this CTA has read the others; they may leave once all have
    __syncthreads();
    k.statistics(a, s, stats + (s.live ? h.q : 0) * s.groups);
#pragma unroll
    for (int i = 0; i < kHeldRows; ++i) {
        const int64_t row = h.row0 + h.lane + i * lay.lanes;
        float f[8], out[8];
        oct_floats(o[i], f);
        if (i < have) {
            k.template apply<DT>(a, f, out);
            oct_store<DT, true>(y, row * a.y_pitch + s.ch0, s.at, oct_round<DT>(out));
        }
        if constexpr (HOLD)
            hold<true>(a, s, f, i < have, row, held);
    }
    if (lay.ranks > 1)
        cluster_wait();
}

// The gradient: a thread keeps dz in fp32 (forming it again would cost the
// activation's special functions twice) and x as it came.
template <int DT, bool BY_OCT, bool HELD>
__global__ void __launch_bounds__(kLayerThreads)
    norm_held_grad_kernel(NormArgs a, const void* dy, Saved x, const void* weight, const void* bias,
                          const float* mean, const float* rstd, void* dx, float* chan)
{
    extern __shared__ float2 shared[];
    const NormLayout& lay = a.lay;
    NormPlace s = norm_place<true>(a);
    const HeldPlace h = held_place(a, s);
    GradRow<DT, true, HELD> g[kHeldGradRows];
    int have = 0;
#pragma unroll
    for (int i = 0; i < kHeldGradRows; ++i) {
        const int r = h.lane + i * lay.lanes;
        if (s.live && r < h.rows) {
            g[i].load(a, s, dy, x, h.row0 + r);
            have = i + 1;
        }
    }
    Chan<BY_OCT> k;
    k.template params<DT, true>(a, s, weight, bias);
    const int width = s.at.cols, items = lay.samples * s.groups;
    float2* slots = shared;                          // [P][run_cols]
    float2* columns = slots + lay.P * width;         // [samples][run_cols]
    float2* sums = columns + lay.samples * width;    // [samples][groups]: S1, S2 of the part
    float2* stats = sums + items;                    // [samples][groups]: first (mean, rstd), then S1 / M, S2 / M
    for (int i = threadIdx.x; i < items; i += blockDim.x) {
        const int q = i / s.groups;
        const int64_t sample = h.tile * lay.samples + q;
        const int64_t at = sample * a.groups + s.group0 + i - q * s.groups;
        stats[i] = sample < a.n ? make_float2(__ldg(mean + at), __ldg(rstd + at)) : make_float2(0.f, 0.f);
    }
    __syncthreads();
    k.statistics(a, s, stats + (s.live ? h.q : 0) * s.groups);
    float dz[kHeldGradRows][8], sz[8], szx[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        sz[j] = szx[j] = 0.f;
#pragma unroll
    for (int i = 0; i < kHeldGradRows; ++i)
        if (i < have) {
            float fd[8], fx[8], hat[8];
            g[i].floats(a, fd, fx);
            k.template slopes<DT>(a, fd, fx, hat, dz[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sz[j] += dz[i][j];
                szx[j] += dz[i][j] * hat[j];
            }
        }
    add_lanes(s, h.lane, lay.lanes, slots, width, sz, szx);
    if (s.p < lay.P && s.at.ch < s.at.cols && h.lane == 0)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            columns[h.q * width + s.at.ch + j] = make_float2(sz[j], szx[j]);
    __syncthreads();
    for (int q = 0; q < lay.samples; ++q)
        weigh_columns<DT>(a, s, weight, columns + q * width, sums + q * s.groups);
    float* out = chan + static_cast<int64_t>(blockIdx.x) * 2 * a.c + s.ch0;
    for (int ch = threadIdx.x; ch < width; ch += blockDim.x) {
        float2 v = columns[ch];
        for (int q = 1; q < lay.samples; ++q) {
            v.x += columns[q * width + ch].x;
            v.y += columns[q * width + ch].y;
        }
        out[ch] = v.y;
        out[a.c + ch] = v.x;
    }
    if (lay.ranks > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    const float m = static_cast<float>(a.l) * static_cast<float>(a.per_group);
    for (int i = threadIdx.x; i < items; i += blockDim.x) {
        float2 v = sums[i];
        if (lay.ranks > 1) {
            v = make_float2(0.f, 0.f);
            for (int r = 0; r < lay.ranks; ++r) {
                const float2 u = cluster_pair(&sums[i], r);
                v.x += u.x;
                v.y += u.y;
            }
        }
        stats[i] = make_float2(v.x / m, v.y / m);
    }
    if (lay.ranks > 1)
        cluster_arrive();
    __syncthreads();
    float s1[BY_OCT ? 1 : 8], s2[BY_OCT ? 1 : 8];
#pragma unroll
    for (int j = 0; j < (BY_OCT ? 1 : 8); ++j) {
        const int ch = s.at.ch + j;
        const float2 t = stats[(s.live ? h.q : 0) * s.groups + (ch < s.at.cols ? local_group(a, ch) : 0)];
        s1[j] = t.x;
        s2[j] = t.y;
    }
#pragma unroll
    for (int i = 0; i < kHeldGradRows; ++i)
        if (i < have) {
            float fx[8], out8[8];
            g[i].saved_floats(a, fx);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                out8[j] = k.rs(j) * (dz[i][j] * k.w[j] - s1[BY_OCT ? 0 : j] -
                                     (fx[j] - k.mu(j)) * k.rs(j) * s2[BY_OCT ? 0 : j]);
            oct_store<DT, true>(dx, (h.row0 + h.lane + i * lay.lanes) * a.x_pitch + s.ch0, s.at,
                                oct_round<DT>(out8));
        }
    if (lay.ranks > 1)
        cluster_wait();
}

template <class K, class... Args>
cudaError_t launch_ranks(K kernel, const NormArgs& a, size_t smem, cudaStream_t st, Args... args)
{
    const void* fn = reinterpret_cast<const void*>(kernel);
    cudaError_t e = cudaSuccess;
    if (a.lay.ranks > 8)
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && smem > 48 * 1024)
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned((a.n + a.lay.samples - 1) / a.lay.samples * a.lay.ranks), unsigned(a.lay.runs));
    cfg.blockDim = dim3(unsigned(a.lay.threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = unsigned(a.lay.ranks);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = a.lay.ranks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a, args...);
}

}  // namespace

#define TSX_BY_HELD(dtype, by_oct, CALL)                            \
    do {                                                            \
        if ((dtype) == TSX_F16) {                                   \
            if (by_oct) { CALL(TSX_F16, true); }                    \
            else { CALL(TSX_F16, false); }                          \
        } else if ((dtype) == TSX_BF16) {                           \
            if (by_oct) { CALL(TSX_BF16, true); }                   \
            else { CALL(TSX_BF16, false); }                         \
        } else {                                                    \
            if (by_oct) { CALL(TSX_F32, true); }                    \
            else { CALL(TSX_F32, false); }                          \
        }                                                           \
    } while (0)

cudaError_t launch_norm_held(int dtype, const NormArgs& a, const void* x, const void* weight, const void* bias, void* y,
                             float* mean, float* rstd, HeldOut held, cudaStream_t st)
{
    const NormLayout& lay = a.lay;
    const size_t width = lay.oct_in_group ? lay.run_cols / 8 : lay.run_cols;
    const size_t smem = ((lay.P + lay.samples) * width + 2 * size_t(lay.samples) * lay.run_groups) * sizeof(float2) +
                        lay.P * sizeof(float);
    cudaError_t e = cudaSuccess;
#define CALL(DT, BY_OCT)                                                                                    \
    e = held.q ? launch_ranks(norm_held_kernel<DT, BY_OCT, true>, a, smem, st, x, weight, bias, y, mean,    \
                              rstd, held)                                                                   \
               : launch_ranks(norm_held_kernel<DT, BY_OCT, false>, a, smem, st, x, weight, bias, y, mean,   \
                              rstd, held)
    TSX_BY_HELD(dtype, lay.oct_in_group, CALL);
#undef CALL
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_norm_held_backward(int dtype, const NormArgs& a, const void* dy, Saved x, const void* weight,
                                      const void* bias, const float* mean, const float* rstd, void* dx,
                                      float* dweight, float* dbias, NormScratch scratch, cudaStream_t st)
{
    const NormLayout& lay = a.lay;
    const size_t smem =
        (size_t(lay.P + lay.samples) * lay.run_cols + 2 * size_t(lay.samples) * lay.run_groups) * sizeof(float2);
    cudaError_t e = cudaSuccess;
#define CALL(DT, BY_OCT)                                                                                      \
    e = x.q ? launch_ranks(norm_held_grad_kernel<DT, BY_OCT, true>, a, smem, st, dy, x, weight, bias, mean,   \
                           rstd, dx, scratch.chan)                                                            \
            : launch_ranks(norm_held_grad_kernel<DT, BY_OCT, false>, a, smem, st, dy, x, weight, bias, mean,  \
                           rstd, dx, scratch.chan)
    TSX_BY_HELD(dtype, lay.oct_in_group, CALL);
#undef CALL
    if (e == cudaSuccess)
        e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    const int64_t slices = (a.n + lay.samples - 1) / lay.samples * lay.ranks;
    return launch_norm_params(a, slices, scratch.chan, dweight, dbias, st);
}

}  // namespace tsx
