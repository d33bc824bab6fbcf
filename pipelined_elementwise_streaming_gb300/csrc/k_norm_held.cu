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

// Which rows a thread holds: lane, lane + lanes, ... of its sample's part.
struct HeldPlace {
    int rank;         // of the cluster's `ranks` CTAs
    int q, lane;      // sample of the CTA, row lane of the sample
    int64_t tile;     // first sample / samples to a CTA
    int64_t sample;
    int64_t row0;     // the part's first row, counted through all samples
    int rows;         // rows of the part
    int mine;         // rows of the thread's lane
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
    h.row0 = h.sample * a.l + h.rank * lay.range;
    h.rows = range_rows(a, lay.range, h.rank);
    h.mine = s.p < lay.P && h.sample < a.n && h.lane < h.rows ? (h.rows - h.lane + lay.lanes - 1) / lay.lanes : 0;
    return h;
}

// all[ranks][items] = every rank's sums; then says that this CTA has read the
// others (they may leave once all have).  After a cluster barrier.
__device__ __forceinline__ void gather_ranks(const float2* sums, int items, int ranks, float2* all)
{
    for (int i = threadIdx.x; i < ranks * items; i += blockDim.x) {
        const int r = i / items;
        all[i] = cluster_pair(sums + i - r * items, r);
    }
    cluster_arrive();
    __syncthreads();
}

template <int DT, bool BY_OCT, bool HOLD, int ROWS>
__global__ void __launch_bounds__(kNormThreads, 2)
    norm_held_kernel(NormArgs a, const void* x, const void* weight, const void* bias, void* y, float* mean,
                     float* rstd, HeldOut held)
{
    extern __shared__ float4 shared4[];
    const NormLayout& lay = a.lay;
    NormPlace s = norm_place<true>(a);
    const HeldPlace h = held_place(a, s);
    Oct<DT> o[ROWS];
    const int have = h.mine;
    load_rows<DT, true>(walk<DT>(x, h.row0 + h.lane, lay.lanes, a.x_pitch, s), s.at, s.live ? have : 0, o);
    Affine k;
    k.template params<DT, true>(a, s, weight, bias);

    const int width = run_width<BY_OCT>(s), stride = slot_stride(width), items = lay.samples * s.groups;
    float4* spare = shared4;                                                // [warps]
    float2* sums = reinterpret_cast<float2*>(spare + kNormThreads / 32);    // [samples][groups]: (mean, M2) of the part
    float2* stats = sums + items;                                           // [samples][groups]: (mean, rstd)
    float2* slots = stats + items;                                          // [P][stride]; then [ranks][items]
    Triples<BY_OCT> t;
    t.clear();
    if (s.live)
        t.add_octs(o, have);
    if (s.p < lay.P && s.at.ch < s.at.cols)   // absent samples leave zeros
        t.leave(s.at, slots + s.p * stride);
    __syncthreads();
    join_groups(slots, stride, lay.samples, s.groups, lay.lanes, a.per_group / (BY_OCT ? 8 : 1), h.rows,
                BY_OCT ? 8.f : 1.f, sums, spare);
    if (lay.ranks > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (lay.ranks > 1)
        gather_ranks(sums, items, lay.ranks, slots);
    const float m = static_cast<float>(a.l) * static_cast<float>(a.per_group);
    for (int i = threadIdx.x; i < items; i += blockDim.x) {
        float2 v = sums[i];
        if (lay.ranks > 1) {
            Triples<true> j;
            j.clear();
            for (int r = 0; r < lay.ranks; ++r) {
                const float2 u = slots[r * items + i];
                const float mu[1] = {u.x}, dev[1] = {u.y};
                j.join(static_cast<float>(range_rows(a, lay.range, r)) * a.per_group, mu, dev);
            }
            v = make_float2(j.mean[0], j.m2[0]);
        }
        v.y = rstd_of(v.y, 1.f / m, a.eps);
        stats[i] = v;
        const int q = lay.samples == 1 ? 0 : i / s.groups;
        const int64_t sample = h.tile * lay.samples + q;
        if (h.rank == 0 && sample < a.n) {
            mean[sample * a.groups + s.group0 + i - q * s.groups] = v.x;
            rstd[sample * a.groups + s.group0 + i - q * s.groups] = v.y;
        }
    }
    __syncthreads();
    k.template statistics<BY_OCT>(a, s, stats + (s.live ? h.q : 0) * s.groups);
    const WalkOut out = walk_out<DT>(y, h.row0 + h.lane, lay.lanes, a.y_pitch, s);
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
        if (s.live && i < have) {
            float2 f[4], v[4];
            oct_floats(o[i], f);
            k.apply(a.act, f, v);
            oct_store<DT, true>(out.p + i * out.step, s.at, oct_round<DT>(v));
        }
    if constexpr (HOLD) {
        HeldPtr to(held, h.row0 + h.lane, lay.lanes, a.c, a.blocks, s.ch0 + s.at.ch, a.block);
#pragma unroll
        for (int i0 = 0; i0 < ROWS; i0 += 4) {
            const Oct<DT> four[4] = {o[i0], o[i0 + 1], o[i0 + 2], o[i0 + 3]};
            if (i0 < have)
                hold_rows<DT, true>(four, have - i0, s.live, s.at, lay.team, a.form, to);
            to.advance(4);
        }
    }
    if (lay.ranks > 1)
        cluster_wait();
}

// The gradient: a thread keeps dz in fp32 (forming it again would cost the
// activation's special functions twice) and x as it came.
template <int DT, bool BY_OCT, bool HELD>
__global__ void __launch_bounds__(kNormThreads, 2)
    norm_held_grad_kernel(NormArgs a, const void* dy, Saved x, const void* weight, const void* bias,
                          const float* mean, const float* rstd, void* dx, float* chan)
{
    extern __shared__ float2 shared[];
    const NormLayout& lay = a.lay;
    NormPlace s = norm_place<true>(a);
    const HeldPlace h = held_place(a, s);
    GradRow<DT, true, HELD> g[kHeldGradRows];
    const int have = s.live ? h.mine : 0;
    const GradWalk<DT, true, HELD> w(a, s, dy, x, h.row0 + h.lane, lay.lanes);
#pragma unroll
    for (int i = 0; i < kHeldGradRows; ++i)
        if (i < have)
            g[i].load(a, s, w, i);
    Chan<BY_OCT> k;
    k.template params<DT, true>(a, s, weight, bias);
    const int width = s.at.cols, stride = slot_stride(width), items = lay.samples * s.groups;
    float2* sums = shared;                           // [samples][groups]: S1, S2 of the part
    float2* stats = sums + items;                    // [samples][groups]: (mean, rstd), then -S1 / M, -S2 / M
    float2* work = stats + items;                    // [threads]
    float2* columns = work + kNormThreads;           // [samples][width]
    float2* slots = columns + lay.samples * width;   // [P][stride]; then [ranks][items]
    let_next_start();
    for (int i = threadIdx.x; i < items; i += blockDim.x) {
        const int q = lay.samples == 1 ? 0 : i / s.groups;
        const int64_t sample = h.tile * lay.samples + q;
        const int64_t at = sample * a.groups + s.group0 + i - q * s.groups;
        stats[i] = sample < a.n ? make_float2(__ldg(mean + at), __ldg(rstd + at)) : make_float2(0.f, 0.f);
    }
    __syncthreads();
    k.statistics(a, s, stats + (s.live ? h.q : 0) * s.groups);
    float2 dz[kHeldGradRows][4], sz[4], szx[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        sz[j] = szx[j] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kHeldGradRows; ++i)
        if (i < have) {
            float2 fd[4], hat[4];
            oct_floats(g[i].dy, fd);
            g[i].hats(a, k, hat);
            k.slopes(a, fd, hat, dz[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sz[j] = __fadd2_rn(sz[j], dz[i][j]);
                szx[j] = __ffma2_rn(dz[i][j], hat[j], szx[j]);
            }
        }
    if (s.p < lay.P && s.at.ch < s.at.cols)
        leave_sums(s.at, sz, szx, slots + s.p * stride);
    __syncthreads();
    sum_lanes(slots, stride, lay.samples, lay.lanes, width, columns, work);
    weigh_columns<DT>(a, s, lay.samples, width, weight, columns, sums);
    float* out = chan + static_cast<int64_t>(blockIdx.x) * 2 * a.c + s.ch0;
    for (int ch = threadIdx.x; ch < width; ch += blockDim.x) {
        float2 v = columns[ch];
        for (int q = 1; q < lay.samples; ++q)
            v = __fadd2_rn(v, columns[q * width + ch]);
        out[ch] = v.y;
        out[a.c + ch] = v.x;
    }
    if (lay.ranks > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (lay.ranks > 1)
        gather_ranks(sums, items, lay.ranks, slots);
    const float m = -static_cast<float>(a.l) * static_cast<float>(a.per_group);
    for (int i = threadIdx.x; i < items; i += blockDim.x) {
        float2 v = sums[i];
        if (lay.ranks > 1) {
            v = slots[i];
            for (int r = 1; r < lay.ranks; ++r)
                v = __fadd2_rn(v, slots[r * items + i]);
        }
        stats[i] = make_float2(v.x / m, v.y / m);
    }
    __syncthreads();
    Gradient<BY_OCT> grad;
    grad.set(a, s, k, stats + (s.live ? h.q : 0) * s.groups);
    const WalkOut to = walk_out<DT>(dx, h.row0 + h.lane, lay.lanes, a.x_pitch, s);
#pragma unroll
    for (int i = 0; i < kHeldGradRows; ++i)
        if (i < have) {
            float2 hat[4], res[4];
            g[i].hats(a, k, hat);
            grad.of(dz[i], hat, res);
            oct_store<DT, true>(to.p + i * to.step, s.at, oct_round<DT>(res));
        }
    if (lay.ranks > 1)
        cluster_wait();
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

namespace {

// Pairs of shared memory for the columns, which the ranks' sums reuse.
size_t slot_pairs(const NormLayout& lay, int width)
{
    const size_t slots = size_t(lay.P) * slot_stride(width);
    const size_t all = lay.ranks > 1 ? size_t(lay.ranks) * lay.samples * lay.run_groups : 0;
    return slots > all ? slots : all;
}

}  // namespace

cudaError_t launch_norm_held(int dtype, const NormArgs& a, const void* x, const void* weight, const void* bias, void* y,
                             float* mean, float* rstd, HeldOut held, cudaStream_t st)
{
    const NormLayout& lay = a.lay;
    const dim3 grid(unsigned((a.n + lay.samples - 1) / lay.samples * lay.ranks), unsigned(lay.runs));
    const int width = lay.oct_in_group ? lay.run_cols / 8 : lay.run_cols;
    const size_t smem = kNormThreads / 32 * sizeof(float4) +
                        (2 * size_t(lay.samples) * lay.run_groups + slot_pairs(lay, width)) * sizeof(float2);
    cudaError_t e = cudaSuccess;
#define CALL(DT, BY_OCT)                                                                                            \
    e = held.q ? launch_grid(norm_held_kernel<DT, BY_OCT, true, kHeldRows>, grid, lay.threads, smem, lay.ranks, false, st, \
                             a, x, weight, bias, y, mean, rstd, held)                                               \
               : launch_grid(norm_held_kernel<DT, BY_OCT, false, kHeldRows>, grid, lay.threads, smem, lay.ranks, false, \
                             st, a, x, weight, bias, y, mean, rstd, held)
    TSX_BY_HELD(dtype, lay.oct_in_group, CALL);
#undef CALL
    return e;
}

cudaError_t launch_norm_held_backward(int dtype, const NormArgs& a, const void* dy, Saved x, const void* weight,
                                      const void* bias, const float* mean, const float* rstd, void* dx,
                                      float* dweight, float* dbias, NormScratch scratch, cudaStream_t st)
{
    const NormLayout& lay = a.lay;
    const int64_t slices = (a.n + lay.samples - 1) / lay.samples * lay.ranks;
    const dim3 grid(unsigned(slices), unsigned(lay.runs));
    const size_t smem = (2 * size_t(lay.samples) * lay.run_groups + kNormThreads +
                         size_t(lay.samples) * lay.run_cols + slot_pairs(lay, lay.run_cols)) *
                        sizeof(float2);
    cudaError_t e = cudaSuccess;
#define CALL(DT, BY_OCT)                                                                                           \
    e = x.q ? launch_grid(norm_held_grad_kernel<DT, BY_OCT, true>, grid, lay.threads, smem, lay.ranks, false, st, a, dy, \
                          x, weight, bias, mean, rstd, dx, scratch.chan)                                           \
            : launch_grid(norm_held_grad_kernel<DT, BY_OCT, false>, grid, lay.threads, smem, lay.ranks, false, st, a, dy, \
                          x, weight, bias, mean, rstd, dx, scratch.chan)
    TSX_BY_HELD(dtype, lay.oct_in_group, CALL);
#undef CALL
    if (e != cudaSuccess)
        return e;
    return launch_norm_params(a, slices, scratch.chan, dweight, dbias, st);
}

}  // namespace tsx
