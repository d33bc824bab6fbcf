// Attention over a paged cache for few rows to a head: single new tokens above all.
//
// Keys and values are read once, and for a handful of rows that is all there is
// to do in earnest: HBM bounds it.  A CTA's four warps work for themselves, each
// on 16 of the 64 keys of a step, with a queue of its own in shared memory that
// it fills by cp.async (a page may start anywhere, so each row of 16-byte chunks
// has its own address) and empties with no barrier but its own.  The products are
// mma.m16n8k16 with the rows as M: up to 16 queries of a key, most of whose places
// stay empty, but that is not what bounds it.
// Scores stay in registers: the accumulators of q k^T are the operand of the
// product with v.  Running maxima and sums are the warp's own; they and the four
// sums of values are joined once at the end of a piece.
//
// In the product with v a weight rounded into the element type loses up to 2^-8 (bf16)
// or 2^-11 of itself, which shows beside the result's own rounding (relative to the
// result's norm 2.0e-3 in place of 1.66e-3 for bf16).  So tiles are of 8 rows where no
// head has more: the other 8 rows of the instruction then take what rounding has left
// of the weights, and 2^-16 or 2^-22 is lost, with the same instructions.  The two sums
// are added at the end of a piece.  9 to 16 rows fill the instruction, and rests in a
// second product took 2 to 8 % longer and made infinite values NaN: weights are rounded
// there, as in the kernel for many rows.
//
// Measured on GB300, GPU time of a call in a CUDA graph over inputs that take turns;
// in parentheses the time of the bytes at the 6791 GB/s of a copy.  One new token to
// each of 64 sequences of 1000 to 16384, bf16, 32 heads over 8 of 128, pages of 16: 217
// to 224 us (213) from one machine to the next; 256 channels 487 (427), 136 490 (227): such
// heads are handled as 256.  One sequence of 100003 keys, f16, 16 heads over 2 of 64: 22.3
// (7.5), of which the join of 152 parts a head takes 7 and a CTA's start, first pages and
// end 5.  16 sequences up to 4096: 22.7 (12.6); one of 300: 9.8.  Queues of three stages
// of 8 KB a warp keep 128 KB of an SM on their way; of 64 channels the stages are half as
// large and there are six.

#include "tsx_attend.cuh"
#include "tsx_device.cuh"

namespace tsx {
namespace {

using namespace dev;

constexpr int kKeys = 64, kWarpKeys = 16, kThreads = 128;
// Stages of a warp's queue: as many bytes on their way for either width.
template <int D>
TSX_HD constexpr int stages() { return D == 64 ? 6 : 3; }
constexpr int kJoinRows = 4, kJoinWarps = 8;
// What a tile costs beside its steps, in steps, and units to a CTA at least: 16
// sequences of up to 4096 keys, 32 heads over 8, 24.8 us with 0, 22.5 with 3, 23.5 with
// 6; four of up to 1000 10.0 us in runs of at least 4, 10.7 of 5, 11.8 of 7.
constexpr int kCost = 3;
constexpr int64_t kLeast = 4;

template <int D>
TSX_HD constexpr int stage_bytes() { return 2 * kWarpKeys * D * 2; }
// Shared memory: the queues, the warps' statistics, the words of run_of.
template <int D>
TSX_HD constexpr int queue_bytes() { return 4 * stages<D>() * stage_bytes<D>(); }
constexpr int kStatsBytes = 4 * 16 * 8, kSumsBytes = (kThreads / 32 + 3) * 8;

__device__ __forceinline__ void ldmatrix(uint32_t at, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t at, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

template <int DT>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (DT == TSX_BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A stage: keys then values, 16 rows of D / 8 chunks of 16 bytes, chunk c of row
// r at place c ^ (r & 7) so that ldmatrix meets every bank once.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk)
{
    return static_cast<uint32_t>(row * (D * 2) + ((chunk ^ (row & 7)) * 16));
}

template <int DT>
__device__ __forceinline__ float value_of(uint16_t w)
{
    return DT == TSX_BF16 ? __uint_as_float(static_cast<uint32_t>(w) << 16) : __half2float(__ushort_as_half(w));
}

// A warp's 16 keys of the next steps of a piece: where each lies, one step ahead
// of its use (key lane % 16 to a lane).
struct Keys {
    int position;   // of the lane's key in the step to come
    int limit;      // keys before this one are wanted
    int page;       // read ahead, -1 if there is none
    const int32_t* pages;

    __device__ __forceinline__ void look(const AttendArgs& a)
    {
        page = position < limit ? pages[page_of(a.paged, position)] : -1;
    }
};

template <int DT, int D>
__device__ __forceinline__ uint32_t load_step(const AttendArgs& a, const Keys& k, int64_t head_at, uint32_t stage)
{
    const int lane = threadIdx.x & 31;
    const bool there = k.page >= 0 && k.page < a.paged.cache_pages;
    const int slot = k.position - page_of(a.paged, k.position) * a.paged.page_size;
    const int64_t at = there ? (k.page * a.paged.page_pitch + slot * a.slot_pitch + head_at) * 2 : 0;
    const uint32_t seen = __ballot_sync(0xffffffffu, there) & 0xffffu;
    constexpr int kChunks = D / 8, kTurns = kWarpKeys * kChunks / 32;
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int id = i * 32 + lane, row = id / kChunks, chunk = id % kChunks;
        const int64_t from = __shfl_sync(0xffffffffu, at, row) + chunk * 16;
        const uint32_t bytes = (seen >> row & 1) && chunk * 8 < a.dim ? 16 : 0;
        const uint32_t to = stage + chunk_at<D>(row, chunk);
        cp_async(to, bytes ? a.k + from : a.k, 16, bytes);
        cp_async(to + kWarpKeys * D * 2, bytes ? a.v + from : a.v, 16, bytes);
    }
    return seen;
}

// M: rows of a tile, 8 or 16.  A thread has row g of them and, of 16, row g + 8.
template <int DT, int D, int M>
__global__ void __launch_bounds__(kThreads, D == 256 ? 1 : 2) attend_kernel(const __grid_constant__ AttendArgs a)
{
    constexpr int kMine = M / 8;
    extern __shared__ __align__(128) unsigned char memory[];
    float2(*stats)[M] = reinterpret_cast<float2(*)[M]>(memory + queue_bytes<D>());
    int64_t* sums = reinterpret_cast<int64_t*>(memory + queue_bytes<D>() + kStatsBytes);
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g = lane / 4, c2 = lane % 4 * 2;
    constexpr int kStages = stages<D>(), kFours = fold_fours(false, D);
    static_assert(kThreads == fold_threads(false), "a row of folded sums to each thread");
    constexpr float kLift = lift<DT, 0>();
    const uint32_t queue = smem_addr(memory) + warp * (kStages * stage_bytes<D>());
    let_next_start();
    Run run = run_of<M, kKeys, kCost, kThreads>(a, kLeast, sums);
    Tail tail{};
    while (run.from < run.to) {
        const Piece p = piece_of<M, kKeys, kCost>(a, run);
        if (p.empty())
            break;   // the run's last units, before a tile's first step
        const int row0 = p.tile * M;
        const int64_t head_at = p.head * a.head_pitch;
        // queries, as the A operand: rows g and g + 8
        uint32_t q[D / 16][4] = {};
#pragma unroll
        for (int half = 0; half < kMine; ++half) {
            const int row = g + half * 8;
            const char* from = a.q + row_at(a, p.seq.first, p.head, row0 + row, a.q_pitch, a.q_head) * 2;
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int ch = k * 16 + e * 8 + c2;
                    q[k][half + 2 * e] =
                        row < p.rows && ch < a.dim ? *reinterpret_cast<const uint32_t*>(from + ch * 2) : 0u;
                }
        }
        int limits[kMine];
#pragma unroll
        for (int r = 0; r < kMine; ++r)
            limits[r] = row_limit(a, p.seq, row0 + g + 8 * r);
        const int first_limit = row_limit(a, p.seq, row0);
        const int last_limit = row_limit(a, p.seq, row0 + p.rows - 1);
        Keys keys;
        keys.limit = min(last_limit, p.seq.length);
        keys.pages = a.paged.pages + p.b * a.paged.pages_pitch;
        keys.position = p.step * kKeys + warp * kWarpKeys + lane % 16;
        keys.look(a);
        uint32_t seen[kStages];
        const int steps = p.end - p.step;
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            seen[i] = 0;
            if (i < steps) {
                seen[i] = load_step<DT, D>(a, keys, head_at, queue + i * stage_bytes<D>());
                keys.position += kKeys;
                keys.look(a);
            }
            cp_async_commit();
        }
        float out[D / 8][4], top[kMine], sum[kMine];
#pragma unroll
        for (int r = 0; r < kMine; ++r) {
            top[r] = -INFINITY;
            sum[r] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                out[i][e] = 0.f;
        int next_in = kStages - 1, next_out = 0;
        int base = p.step * kKeys + warp * kWarpKeys;
        // what has been folded (see kFold) added to the sums; then `each` of them may be put away
        float4* const folded = folded_at<kThreads, kFours>(a);
        const auto fold = [&](bool first, auto&& each) {
            float4 held = make_float4(0.f, -INFINITY, 0.f, -INFINITY);
            if (!first)
                held = folded[kFours * kThreads];
            const float now[2] = {reference(top[0], kLift), reference(top[kMine - 1], kLift)};
            const float f[2] = {refer(held.y, now[0]), M == 8 ? refer(held.y, now[0]) : refer(held.w, now[1])};
            sum[0] += held.x * f[0];
            if constexpr (M == 16)
                sum[1] += held.z * f[1];
#pragma unroll
            for (int i = 0; i < kFours; ++i) {
                if (!first) {
                    const float4 g = folded[i * kThreads];
                    out[i][0] += g.x * f[0];
                    out[i][1] += g.y * f[0];
                    out[i][2] += g.z * f[1];
                    out[i][3] += g.w * f[1];
                }
                each(i);
            }
        };
        for (int step = 0; step < steps; ++step, base += kKeys) {
            if (step > 0 && step % kFold == 0) {
                fold(step == kFold, [&](int i) {
                    folded[i * kThreads] = make_float4(out[i][0], out[i][1], out[i][2], out[i][3]);
                    out[i][0] = out[i][1] = out[i][2] = out[i][3] = 0.f;
                });
                folded[kFours * kThreads] = make_float4(sum[0], reference(top[0], kLift), sum[kMine - 1],
                                                        reference(top[kMine - 1], kLift));
#pragma unroll
                for (int r = 0; r < kMine; ++r)
                    sum[r] = 0.f;
            }
            cp_async_wait(kStages - 2);
            __syncwarp();
            const uint32_t mask = seen[0];
#pragma unroll
            for (int i = 0; i + 2 < kStages; ++i)
                seen[i] = seen[i + 1];
            uint32_t more = 0;
            if (step + kStages - 1 < steps) {   // into the stage that the last step has left
                more = load_step<DT, D>(a, keys, head_at, queue + next_in * stage_bytes<D>());
                keys.position += kKeys;
                keys.look(a);
            }
            seen[kStages - 2] = more;
            cp_async_commit();
            const uint32_t stage = queue + next_out * stage_bytes<D>();
            next_in = next_in + 1 == kStages ? 0 : next_in + 1;
            next_out = next_out + 1 == kStages ? 0 : next_out + 1;
            if (mask == 0)
                continue;
            float s[2][4] = {};
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t b[4];
                ldmatrix(stage + chunk_at<D>(lane / 16 * 8 + lane % 8, 2 * k + (lane / 8 & 1)), b);
                mma<DT>(s[0], q[k], b[0], b[1]);
                mma<DT>(s[1], q[k], b[2], b[3]);
            }
            float most[kMine];
#pragma unroll
            for (int r = 0; r < kMine; ++r)
                most[r] = -INFINITY;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2 * kMine; ++e) {
                    const int key = j * 8 + c2 + (e & 1);
                    const bool sees = (mask >> key & 1) && base + key < limits[e >> 1];
                    s[j][e] = sees ? s[j][e] * a.scale_log2 : -INFINITY;
                    most[e >> 1] = fmaxf(most[e >> 1], s[j][e]);
                }
            bool grows = false;
#pragma unroll
            for (int r = 0; r < kMine; ++r) {
                most[r] = fmaxf(most[r], __shfl_xor_sync(0xffffffffu, most[r], 1));
                most[r] = fmaxf(most[r], __shfl_xor_sync(0xffffffffu, most[r], 2));
                most[r] = fmaxf(most[r], top[r]);
                grows |= most[r] != top[r];
            }
            if (__any_sync(0xffffffffu, grows)) {
                float f[kMine];
#pragma unroll
                for (int r = 0; r < kMine; ++r) {   // no score yet: nothing to scale
                    f[r] = top[r] == -INFINITY ? 1.f
                                               : exp2_fast(reference(top[r], kLift) - reference(most[r], kLift));
                    top[r] = most[r];
                    sum[r] *= f[r];
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        out[i][e] *= f[M == 8 ? 0 : e >> 1];
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2 * kMine; ++e) {
                    s[j][e] = exp2_fast(s[j][e] - (top[e >> 1] == -INFINITY ? 0.f : reference(top[e >> 1], kLift)));
                    sum[e >> 1] += s[j][e];
                }
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                w[2 * j] = pack2<DT>(s[j][0], s[j][1]);
                w[2 * j + 1] = M == 16 ? pack2<DT>(s[j][2], s[j][3])
                                       : pack2<DT>(s[j][0] - value_of<DT>(static_cast<uint16_t>(w[2 * j])),
                                                   s[j][1] - value_of<DT>(static_cast<uint16_t>(w[2 * j] >> 16)));
            }
            const uint32_t values = stage + kWarpKeys * D * 2;
            if (base + kWarpKeys > first_limit) {
                // Some row may not see some key: 0 times an infinity of such a value would be NaN.  What is not
                // finite is taken out of the product and added to the rows that see it.
                unsigned char* bytes = memory + (values - smem_addr(memory));
                bool bad = false;
                for (int i = lane; i < kWarpKeys * D / 8; i += 32) {
                    const uint4 v = *reinterpret_cast<const uint4*>(bytes + i * 16);
                    bad |= not_finite<DT>(v.x) || not_finite<DT>(v.y) || not_finite<DT>(v.z) || not_finite<DT>(v.w);
                }
                if (__any_sync(0xffffffffu, bad)) {
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
#pragma unroll 1
                        for (int key = 0; key < kWarpKeys; ++key) {
                            const uint32_t pair = *reinterpret_cast<const uint32_t*>(bytes + chunk_at<D>(key, i) + c2 * 2);
                            if (!not_finite<DT>(pair) || !(mask >> key & 1))
                                continue;
#pragma unroll
                            for (int e = 0; e < 2 * kMine; ++e) {
                                const uint16_t v = static_cast<uint16_t>(e & 1 ? pair >> 16 : pair);
                                if (not_finite<DT>(v) && base + key < limits[e >> 1])
                                    out[i][e] += value_of<DT>(v);
                            }
                        }
                    __syncwarp();
                    for (int i = lane; i < kWarpKeys * D / 2; i += 32) {
                        uint32_t* at = reinterpret_cast<uint32_t*>(bytes) + i;
                        const uint32_t v = *at;
                        if (not_finite<DT>(v))
                            *at = (not_finite<DT>(v & 0xffffu) ? 0u : v & 0xffffu) |
                                  (not_finite<DT>(v >> 16) ? 0u : v & 0xffff0000u);
                    }
                    __syncwarp();
                }
            }
#pragma unroll
            for (int i = 0; i < D / 8; i += 2) {
                uint32_t b[4];
                ldmatrix_trans(values + chunk_at<D>((lane / 8 & 1) * 8 + lane % 8, i + lane / 16), b);
                mma<DT>(out[i], w, b[0], b[1]);
                mma<DT>(out[i + 1], w, b[2], b[3]);
            }
        }
        // the four warps' sums, each relative to its own maximum
        cp_async_wait(0);
        if (steps > kFold)
            fold(false, [](int) {});
        if constexpr (M == 8)
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)   // of an infinite value the rests are not wanted: theirs have any sign
                    out[i][e] += fabsf(out[i][e]) < INFINITY ? out[i][e + 2] : 0.f;
#pragma unroll
        for (int r = 0; r < kMine; ++r) {
            sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
            sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
            if (lane % 4 == 0)
                stats[warp][g + 8 * r] = make_float2(reference(top[r], kLift), sum[r]);
        }
        __syncthreads();   // also: the queues are empty, and their memory free
        float* joined = reinterpret_cast<float*>(memory);   // [4][M][D]
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int r = 0; r < kMine; ++r)
                *reinterpret_cast<float2*>(joined + (warp * M + g + 8 * r) * D + i * 8 + c2) =
                    make_float2(out[i][2 * r], out[i][2 * r + 1]);
        __syncthreads();
        const bool whole = p.whole();
        const int slot = part_slot(p);
        constexpr int kRowFours = D / 4;
        for (int i = threadIdx.x; i < p.rows * kRowFours; i += kThreads) {
            const int row = i / kRowFours, ch = i % kRowFours * 4;
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                m = fmaxf(m, stats[w][row].x);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float2 t = stats[w][row];
                const float f = t.x == -INFINITY ? (t.y != t.y ? t.y : 0.f) : exp2_fast(t.x - m);
                const float4 o = *reinterpret_cast<const float4*>(joined + (w * M + row) * D + ch);
                if (t.x == -INFINITY && t.y == t.y)
                    continue;   // nothing seen
                l += t.y * f;
                v.x += o.x * f;
                v.y += o.y * f;
                v.z += o.z * f;
                v.w += o.w * f;
            }
            if (whole) {
                const float f = l > 0.f || l != l ? 1.f / l : 0.f;
                if (ch < a.dim) {
                    char* to = a.out + (row_at(a, p.seq.first, p.head, row0 + row, a.out_pitch, a.out_head) + ch) * 2;
                    *reinterpret_cast<uint2*>(to) = make_uint2(pack2<DT>(v.x * f, v.y * f), pack2<DT>(v.z * f, v.w * f));
                }
                if (ch == 0)
                    store_lse(a, p.seq.first, p.head, row0 + row, m, l);
            } else {
                *reinterpret_cast<float4*>(a.parts + (static_cast<int64_t>(slot) * M + row) * D + ch) = v;
                if (ch == 0)
                    a.stats[slot * M + row] = make_float2(m, l);
            }
        }
        const Tail t = tail_of<M, kCost>(run, p);
        if (t.per)
            tail = t;
        __syncthreads();   // before the queues are used again
        advance<M>(a, run, p);
    }
    if (threadIdx.x == 0)
        a.tails[blockIdx.x] = tail;
}

template <int DT, int D, int M>
cudaError_t launch_rows(const AttendArgs& a, cudaStream_t st)
{
    const cudaError_t e = launch_grid<attend_kernel<DT, D, M>>(dim3(unsigned(a.ctas)), kThreads,
                                                               queue_bytes<D>() + kStatsBytes + kSumsBytes, 1, false, st, a);
    if (e != cudaSuccess)
        return e;
    return launch_grid<attend_join_kernel<DT, D, M, kJoinRows, kJoinWarps>>(
        dim3(unsigned(a.ctas), M / kJoinRows), kJoinWarps * 32, 0, 1, true, st, a);
}

template <int DT, int M>
cudaError_t launch_dim(const AttendArgs& a, cudaStream_t st)
{
    return a.dim <= 64    ? launch_rows<DT, 64, M>(a, st)
           : a.dim <= 128 ? launch_rows<DT, 128, M>(a, st)
                          : launch_rows<DT, 256, M>(a, st);
}

template <int DT>
cudaError_t launch_few(const AttendArgs& a, int rows, cudaStream_t st)
{
    return rows == 8 ? launch_dim<DT, 8>(a, st) : launch_dim<DT, 16>(a, st);
}

}  // namespace

int attend_few_ctas(int dim) { return dim <= 128 ? 2 * 152 : 152; }

cudaError_t launch_attend_few(int dtype, const AttendArgs& a, int rows, cudaStream_t st)
{
    return dtype == TSX_BF16 ? launch_few<TSX_BF16>(a, rows, st) : launch_few<TSX_F16>(a, rows, st);
}

}  // namespace tsx
