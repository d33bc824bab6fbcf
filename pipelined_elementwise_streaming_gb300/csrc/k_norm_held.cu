// Group norm of samples that fit on chip: a CTA, or a cluster of CTAs that
// share a sample's rows, holds a run of channels of a sample in shared memory,
// so that its operands are read once.
//
// Every thread fills its own slots of shared memory by cp.async and reads them
// back itself, so that no barrier guards them: it asks for a few rows ahead and
// sums those that have come.  The statistics go through the CTA's shared memory
// (tsx_norm.cuh); in a cluster every rank puts its groups' sums into the others'
// memory, and all join them in the same order, so they agree to the bit.  A CTA
// takes several small samples side by side.
//
// What bounds it is the chain: loads, which overlap with the first sums; the
// sums over the row lanes; the cluster's barrier; the second pass over the rows,
// bound by the special-function unit with silu (an exponential and a reciprocal
// an element, 12 cycles of a quarter SM for 32); the stores.  In cycles of a CTA
// of f16 [8, 4096, 320]: 9 to 13 thousand, 4, 2, 8.  Two CTAs to an SM do not
// fill one another's gaps where all of them run side by side.
//
// Measured on GB300, GPU time of a call in a CUDA graph that repeats it on the same
// tensors, for both kinds of kernels; with nothing left in L2 (tensors that take
// turns); HBM's own time at 6786 GB/s:
//                                         held   streaming   held, cold   HBM
//   forward   f16 [8, 4096, 320], 32 groups  14.7   17.6        16.4         6.2
//             bf16 [4, 1024, 1280]            9.2   17.0        10.7         3.1
//             bf16 [256, 256, 512]           32.1   42.2        32.2        19.8
//             fp32 [2000, 64, 256]           44.3   83.5        44.3        38.6
//   gradient  bf16 [4, 1024, 1280]           15.6   19.6        16.8         4.6
//             bf16 [2000, 64, 256]           68.5  109.7        68.5        29.0
// Samples of a row or two, one to a CTA, are far from HBM: what a CTA does once
// outweighs its rows.  Heads of 80 channels, bf16 [8192, 1, 2560] in 32 groups:
// forward 121 us (12.4), gradient 240 (18.5).
// Clusters of 16, or one CTA of 512 threads to an SM, were slower: the SMs hold
// 14 clusters of 16 at two CTAs to an SM, 36 of eight, and a second wave doubles
// the time (bf16 [16, 1024, 640] with its checkpoint 46 us in 16 clusters of
// large CTAs, 21 streaming).

#include "tsx_norm.cuh"

namespace tsx {
namespace {

using namespace dev;

// Rows of a thread to a cp.async group, and groups on their way ahead of the
// one in use.  All rows asked for at once kept the threads from summing (f16 [8,
// 4096, 320] 17.0 us, 15.5 so; forward 2 groups ahead 34.3 us against 32.2 for
// bf16 [256, 256, 512], 4 ahead 16.0 against 15.6 for the first; backward 3
// ahead 77.0 us against 75.4 for [2000, 64, 256]).  Octs that are no vectors are loaded at once: nothing of theirs
// goes on while a thread computes.
constexpr int kAhead = 3, kAskRows = 4, kGradAhead = 2, kGradAskRows = 2;

// Which rows a thread holds: lane, lane + lanes, ... of its sample's part.
struct HeldPlace {
    int rank;         // of the cluster's `ranks` CTAs
    int q, lane;      // sample of the CTA, row lane of the sample
    int64_t tile;     // first sample / samples to a CTA
    int64_t sample;
    int64_t row0;     // the part's first row, counted through all samples
    int rows;         // rows of the part
    int mine;         // rows of the thread's lane
    bool live;        // the thread has channels of a sample that exists
};

__device__ __forceinline__ HeldPlace held_place(const NormArgs& a, const NormPlace& s, int64_t tile)
{
    const NormLayout& lay = a.lay;
    HeldPlace h;
    h.tile = tile;
    h.rank = blockIdx.x % lay.ranks;
    h.q = s.p / lay.lanes;
    h.lane = s.p - h.q * lay.lanes;
    h.sample = h.tile * lay.samples + h.q;
    h.live = s.live && h.sample < a.n;
    h.row0 = h.sample * a.l + h.rank * lay.range;
    h.rows = range_rows(a, lay.range, h.rank);
    h.mine = s.p < lay.P && h.sample < a.n && h.lane < h.rows ? (h.rows - h.lane + lay.lanes - 1) / lay.lanes : 0;
    return h;
}

// all[ranks][items] of every rank = this rank's sums, for all threads of the
// cluster on return.  Called after the sums are there for all threads, and
// after an arrival at the cluster barrier by which every CTA had started.  No
// rank reads another's memory, so none has to wait for another to leave.
__device__ __forceinline__ void share_sums(const float2* sums, int items, int rank, int ranks, float2* all)
{
    cluster_wait();
    for (int i = threadIdx.x; i < ranks * items; i += blockDim.x) {
        const int r = i / items, at = i - r * items;
        cluster_put(all + rank * items + at, r, sums[at]);
    }
    cluster_arrive();
    cluster_wait();
}

// A thread's octs of one operand in shared memory.  Octs that are no vectors
// go through registers.
template <int DT, bool VEC>
struct Slots {
    static constexpr uint32_t kVecs = elem_size(DT) / 2;   // 16-byte vectors of an oct
    uint32_t at, step;   // first oct; from vector to vector
    __device__ __forceinline__ explicit Slots(const char* shared)
        : at(smem_addr(shared) + threadIdx.x * 16), step(blockDim.x * 16)
    {
    }
    // The walk's next N octs, of which n exist, to the places from i on.
    template <int N>
    __device__ __forceinline__ void ask(int i, int n, const Walk& w, const OctAt& oct) const
    {
        if constexpr (VEC) {
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (k < n)
                    oct_async<DT>(at + (i + k) * kVecs * step, step, w.p + k * w.step);
        } else {
            Oct<DT> o[N];
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (k < n)
                    o[k] = oct_load<DT, false>(w.p + k * w.step, oct);
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (k < n)
#pragma unroll
                    for (uint32_t h = 0; h < kVecs; ++h)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + ((i + k) * kVecs + h) * step),
                                     "r"(o[k].w[4 * h]), "r"(o[k].w[4 * h + 1]), "r"(o[k].w[4 * h + 2]),
                                     "r"(o[k].w[4 * h + 3])
                                     : "memory");
        }
    }
    __device__ __forceinline__ Oct<DT> take(int i) const
    {
        Oct<DT> o;
#pragma unroll
        for (uint32_t h = 0; h < kVecs; ++h)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(o.w[4 * h]), "=r"(o.w[4 * h + 1]), "=r"(o.w[4 * h + 2]), "=r"(o.w[4 * h + 3])
                         : "r"(at + (i * kVecs + h) * step));
        return o;
    }
    // Four octs from i on; those past the thread's n rows are zeros.
    __device__ __forceinline__ void take4(int i, int n, Oct<DT> (&o)[4]) const
    {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n)
                o[k] = take(i + k);
            else
                oct_zero(o[k]);
    }
};

template <int DT, bool VEC, bool BY_OCT, bool HOLD>
__global__ void __launch_bounds__(kNormThreads, 2)
    norm_held_kernel(NormArgs a, const void* x, const void* weight, const void* bias, void* y, float* mean,
                     float* rstd, HeldOut held)
{
    extern __shared__ float4 shared4[];
    const NormLayout& lay = a.lay;
    const NormPlace s = norm_place<VEC>(a);
    const HeldPlace h = held_place(a, s, blockIdx.x / lay.ranks);
    const int mine = h.live ? h.mine : 0;
    const int width = run_width<BY_OCT>(s), stride = slot_stride(width), items = lay.samples * s.groups;
    const Slots<DT, VEC> rows(reinterpret_cast<char*>(shared4));
    // [samples][groups]: (mean, M2) of the part; (mean, rstd)
    float2* sums = reinterpret_cast<float2*>(shared4 + Slots<DT, VEC>::kVecs * lay.lane_rows * blockDim.x);
    float2* stats = sums + items;
    float2* all = stats + items;                                    // clusters: [ranks][items]
    float2* slots = all + (lay.ranks > 1 ? lay.ranks * items : 0);   // [P][stride]
    if (lay.ranks > 1)
        cluster_arrive();
    Walk w = walk<DT>(x, h.row0 + h.lane, lay.lanes, a.x_pitch, s);
    auto ask = [&](int i) {
        rows.template ask<kAskRows>(i, mine - i, w, s.at);
        cp_async_commit();
        w.p += kAskRows * w.step;
    };
    const int first = VEC ? kAhead * kAskRows : mine;
    for (int i = 0; i < first; i += kAskRows)
        ask(i);
    Affine<BY_OCT> k;
    k.template params<DT, VEC>(a, s, weight, bias);
    Triples<BY_OCT> t;
    t.clear();
    for (int i = 0; i < mine; i += kAskRows) {
        if constexpr (VEC) {
            ask(i + kAhead * kAskRows);
            cp_async_wait(kAhead);
        }
        Oct<DT> o[4];
        rows.take4(i, mine, o);
        t.add_octs(o, mine - i);
    }
    if (s.p < lay.P && s.at.ch < s.at.cols)   // absent samples leave zeros
        t.leave(s.at, slots + s.p * stride);
    __syncthreads();
    join_groups(lay, slots, stride, lay.samples, s.groups, lay.lanes, a.per_group / (BY_OCT ? 8 : 1), h.rows,
                BY_OCT ? 8.f : 1.f, sums);
    __syncthreads();
    if (lay.ranks > 1)
        share_sums(sums, items, h.rank, lay.ranks, all);
    const float m = static_cast<float>(a.l) * static_cast<float>(a.per_group);
    for (int i = threadIdx.x; i < items; i += blockDim.x) {
        float2 v = sums[i];
        if (lay.ranks > 1)
            v = join_ranges(all + i, items, lay.ranks, static_cast<int>(a.l), static_cast<int>(lay.range),
                            static_cast<float>(a.per_group));
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
    k.statistics(a, s, stats + (h.live ? h.q : 0) * s.groups);
    WalkOut out = walk_out<DT>(y, h.row0 + h.lane, lay.lanes, a.y_pitch, s);
    HeldPtr to;
    if constexpr (HOLD)
        to = HeldPtr(held, h.row0 + h.lane, lay.lanes, a.c, a.blocks, s.ch0 + s.at.ch, a.block);
    const int loop = HOLD ? lay.lane_rows : mine;   // every lane of a warp comes to the checkpoint's shuffles
    for (int i0 = 0; i0 < loop; i0 += 4) {
        Oct<DT> o[4];
        rows.take4(i0, mine, o);
        by_act(a.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 f[4], v[4];
                oct_floats(o[i], f);
                k.apply(act, f, v);
                if (i0 + i < mine)
                    oct_store<DT, VEC>(out.p + i * out.step, s.at, oct_round<DT>(v));
            }
        });
        out.p += 4 * out.step;
        if constexpr (HOLD) {
            hold_rows<DT, VEC>(o, h.live, s.at, lay.team, a.form, HeldRows{to, h.mine - i0});
            to.advance(4);
        }
    }
}

// The gradient.  dz is formed twice rather than held in fp32: the second time
// costs a few instructions an element, the room would halve the rows that a
// CTA holds.  MANY: each CTA takes every gridDim.x-th tile of samples, so that
// dweight and dbias have no more slices than there are CTAs.
template <int DT, bool VEC, bool BY_OCT, bool HELD, bool MANY>
__global__ void __launch_bounds__(kNormThreads, 2)
    norm_held_grad_kernel(NormArgs a, const void* dy, Saved x, const void* weight, const void* bias,
                          const float* mean, const float* rstd, void* dx, float* chan)
{
    extern __shared__ float4 shared4[];
    const NormLayout& lay = a.lay;
    const NormPlace s = norm_place<VEC>(a);
    const int threads = static_cast<int>(blockDim.x);
    const int width = s.at.cols, stride = slot_stride(width), items = lay.samples * s.groups;
    // dy's octs; x's, or the checkpoint's numbers and scales
    const Slots<DT, VEC> rows(reinterpret_cast<char*>(shared4));
    char* second = reinterpret_cast<char*>(shared4 + Slots<DT, VEC>::kVecs * lay.lane_rows * threads);
    const Slots<DT, VEC> xs(second);
    const uint32_t qs = smem_addr(second) + threadIdx.x * 8;
    const uint32_t scales = smem_addr(second) + lay.lane_rows * threads * 8 + threadIdx.x * 4;
    const size_t bytes = size_t(lay.lane_rows) * threads * (HELD ? 12 : 16 * Slots<DT, VEC>::kVecs);
    float2* sums = reinterpret_cast<float2*>(second + bytes);   // [samples][groups]: S1, S2 of the part
    float2* stats = sums + items;                    // [samples][groups]: (mean, rstd), then -S1 / M, -S2 / M
    float2* work = stats + items;                    // [threads]
    float2* columns = work + kNormThreads;           // [samples][width]
    float2* all = columns + lay.samples * width;                     // clusters: [ranks][items]
    float2* slots = all + (lay.ranks > 1 ? lay.ranks * items : 0);   // [P][stride]
    let_next_start();
    if (lay.ranks > 1)
        cluster_arrive();
    const int64_t tiles = (a.n + lay.samples - 1) / lay.samples, tile0 = blockIdx.x / lay.ranks;
    int64_t tile = tile0;
    do {
        const HeldPlace h = held_place(a, s, tile);
        const int mine = h.live ? h.mine : 0;
        const GradWalk<DT, VEC, HELD> walk_rows(a, s, dy, x, h.row0 + h.lane, lay.lanes);
        GradWalk<DT, VEC, HELD> w = walk_rows;
        auto ask = [&](int i) {
            constexpr int N = kGradAskRows;
            rows.template ask<N>(i, mine - i, w.dy, s.at);
            if constexpr (!HELD) {
                xs.template ask<N>(i, mine - i, w.x, s.at);
            } else if constexpr (VEC) {
#pragma unroll
                for (int k = 0; k < N; ++k)
                    if (i + k < mine) {
                        cp_async(qs + (i + k) * threads * 8, w.q + k * w.q_step, 8, 8);
                        cp_async(scales + (i + k) * threads * 4, w.scale + k * w.scale_step, 4, 4);
                    }
            } else {
                Held q[N];
#pragma unroll
                for (int k = 0; k < N; ++k)
                    if (i + k < mine)
                        q[k] = held_load<false>(w.q + k * w.q_step, s.at);
#pragma unroll
                for (int k = 0; k < N; ++k)
                    if (i + k < mine)
                        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(qs + (i + k) * threads * 8), "r"(q[k].w[0]),
                                     "r"(q[k].w[1])
                                     : "memory");
            }
            cp_async_commit();
            w.advance(N);
        };
        const int first = VEC ? kGradAhead * kGradAskRows : mine;
        for (int i = 0; i < first; i += kGradAskRows)
            ask(i);
        // rows i, i + 1, ...; those past the thread's last are zeros
        auto take = [&](int i, GradRow<DT, VEC, HELD>(&g)[kGradAskRows]) {
#pragma unroll
            for (int n = 0; n < kGradAskRows; ++n) {
                if (i + n >= mine) {
                    g[n].clear();
                    continue;
                }
                g[n].dy = rows.take(i + n);
                if constexpr (HELD) {
                    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                 : "=r"(g[n].q.w[0]), "=r"(g[n].q.w[1])
                                 : "r"(qs + (i + n) * threads * 8));
                    if constexpr (VEC)
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(g[n].scale[0]) : "r"(scales + (i + n) * threads * 4));
                    else
                        g[n].load_scales(a, s, walk_rows, i + n);   // one to a channel: again from L1 or L2
                } else {
                    g[n].x = xs.take(i + n);
                }
            }
        };
        Chan<BY_OCT> k;
        k.template params<DT, VEC>(a, s, weight, bias);
        for (int i = threadIdx.x; i < items; i += threads) {
            const int q = lay.samples == 1 ? 0 : i / s.groups;
            const int64_t sample = h.tile * lay.samples + q;
            const int64_t at = sample * a.groups + s.group0 + i - q * s.groups;
            stats[i] = sample < a.n ? make_float2(__ldg(mean + at), __ldg(rstd + at)) : make_float2(0.f, 0.f);
        }
        __syncthreads();
        k.statistics(a, s, stats + (h.live ? h.q : 0) * s.groups);
        float2 sz[4], szx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sz[j] = szx[j] = make_float2(0.f, 0.f);
        for (int i0 = 0; i0 < mine; i0 += kGradAskRows) {
            if constexpr (VEC) {
                ask(i0 + kGradAhead * kGradAskRows);
                cp_async_wait(kGradAhead);
            }
            GradRow<DT, VEC, HELD> g[kGradAskRows];
            take(i0, g);
            by_act(a.act, [&](auto act) {
#pragma unroll
                for (int i = 0; i < kGradAskRows; ++i) {
                    float2 fd[4], hat[4], dz[4];
                    oct_floats(g[i].dy, fd);
                    g[i].hats(a.form, k, hat);
                    k.slopes(act, fd, hat, dz);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sz[j] = __fadd2_rn(sz[j], dz[j]);
                        szx[j] = __ffma2_rn(dz[j], hat[j], szx[j]);
                    }
                }
            });
        }
        if (s.p < lay.P && s.at.ch < s.at.cols)
            leave_sums(s.at, sz, szx, slots + s.p * stride);
        __syncthreads();
        sum_lanes(slots, stride, lay.samples, lay.lanes, width, columns, work);
        weigh_columns<DT>(a, s, lay.samples, width, weight, columns, sums);
        add_slice(chan, a.c, s.ch0, width, MANY && tile != tile0, [&](int ch) {
            float2 v = columns[ch];
            for (int q = 1; q < lay.samples; ++q)
                v = __fadd2_rn(v, columns[q * width + ch]);
            return v;
        });
        __syncthreads();
        if (lay.ranks > 1)
            share_sums(sums, items, h.rank, lay.ranks, all);
        const float m = -static_cast<float>(a.l) * static_cast<float>(a.per_group);
        for (int i = threadIdx.x; i < items; i += threads) {
            float2 v = sums[i];
            if (lay.ranks > 1) {
                v = all[i];
                for (int r = 1; r < lay.ranks; ++r)
                    v = __fadd2_rn(v, all[r * items + i]);
            }
            stats[i] = make_float2(v.x / m, v.y / m);
        }
        __syncthreads();
        Gradient<BY_OCT> grad;
        grad.set(a, s, k, stats + (h.live ? h.q : 0) * s.groups);
        WalkOut to = walk_out<DT>(dx, h.row0 + h.lane, lay.lanes, a.x_pitch, s);
        for (int i0 = 0; i0 < mine; i0 += kGradAskRows) {
            GradRow<DT, VEC, HELD> g[kGradAskRows];
            take(i0, g);
            by_act(a.act, [&](auto act) {
#pragma unroll
                for (int i = 0; i < kGradAskRows; ++i) {
                    float2 fd[4], hat[4], dz[4], res[4];
                    oct_floats(g[i].dy, fd);
                    g[i].hats(a.form, k, hat);
                    k.slopes(act, fd, hat, dz);
                    grad.of(k, dz, hat, res);
                    if (i0 + i < mine)
                        oct_store<DT, VEC>(to.p + i * to.step, s.at, oct_round<DT>(res));
                }
            });
            to.p += kGradAskRows * to.step;
        }
        if constexpr (MANY) {
            tile += gridDim.x;   // no cluster
            __syncthreads();     // stats are read
        }
    } while (MANY && tile < tiles);
}

}  // namespace

size_t held_bytes(const NormLayout& lay, int es, bool backward, bool held)
{
    const size_t octs = size_t(lay.lane_rows) * lay.threads;
    const size_t items = size_t(lay.samples) * lay.run_groups;
    const int width = !backward && lay.oct_in_group ? lay.run_cols / 8 : lay.run_cols;
    size_t pairs = 2 * items + size_t(lay.P) * slot_stride(width);
    if (lay.ranks > 1)
        pairs += size_t(lay.ranks) * items;
    if (backward)
        pairs += kNormThreads + size_t(lay.samples) * width;
    return octs * es * 8 + (backward ? octs * (held ? 12 : es * 8) : 0) + pairs * sizeof(float2);
}

cudaError_t launch_norm_held(int dtype, const NormArgs& a, const void* x, const void* weight, const void* bias, void* y,
                             float* mean, float* rstd, HeldOut held, cudaStream_t st)
{
    const NormLayout& lay = a.lay;
    const dim3 grid(unsigned((a.n + lay.samples - 1) / lay.samples * lay.ranks), unsigned(lay.runs));
    const size_t smem = held_bytes(lay, elem_size(dtype), false, false);
    cudaError_t e = cudaSuccess;
#define CALL(DT, VEC, BY_OCT)                                                                                            \
    e = held.q ? launch_grid<norm_held_kernel<DT, VEC, BY_OCT, true>>(grid, lay.threads, smem, lay.ranks, false, st, \
                             a, x, weight, bias, y, mean, rstd, held)                                               \
               : launch_grid<norm_held_kernel<DT, VEC, BY_OCT, false>>(grid, lay.threads, smem, lay.ranks, false, \
                             st, a, x, weight, bias, y, mean, rstd, held)
    TSX_BY_LAYOUT(dtype, lay, CALL);
#undef CALL
    return e;
}

cudaError_t launch_norm_held_backward(int dtype, const NormArgs& a, const void* dy, Saved x, const void* weight,
                                      const void* bias, const float* mean, const float* rstd, void* dx,
                                      float* dweight, float* dbias, NormScratch scratch, cudaStream_t st)
{
    const NormLayout& lay = a.lay;
    const dim3 grid(unsigned(lay.slices), unsigned(lay.runs));
    const size_t smem = held_bytes(lay, elem_size(dtype), true, x.q != nullptr);
    cudaError_t e = cudaSuccess;
    const bool many = lay.slices < (a.n + lay.samples - 1) / lay.samples * lay.ranks;
#define KERNEL(DT, VEC, BY_OCT, HELD, MANY)                                                                            \
    launch_grid<norm_held_grad_kernel<DT, VEC, BY_OCT, HELD, MANY>>(grid, lay.threads, smem, lay.ranks, false, st, a,  \
                                                                    dy, x, weight, bias, mean, rstd, dx, scratch.chan)
#define CALL(DT, VEC, BY_OCT)                                                                                          \
    e = x.q ? (many ? KERNEL(DT, VEC, BY_OCT, true, true) : KERNEL(DT, VEC, BY_OCT, true, false))                      \
            : (many ? KERNEL(DT, VEC, BY_OCT, false, true) : KERNEL(DT, VEC, BY_OCT, false, false))
    TSX_BY_LAYOUT(dtype, lay, CALL);
#undef CALL
#undef KERNEL
    if (e != cudaSuccess)
        return e;
    return launch_norm_params(a, lay.slices, scratch.chan, dweight, dbias, st);
}

}  // namespace tsx
