// Gated activation h = act(gate) * up and its gradient, and the packing of
// activations into 8 bits and back.
//
// All of them are one pass over their operands with a few to a few dozen
// instructions an element, so HBM bounds them.  A thread keeps its eight
// channels and loads a few rows before it uses the first, so that enough bytes
// are in flight without a ring in shared memory; CTAs live for those rows only,
// as many as the tensor has.  Formulas, with p the sigmoid of the activation:
//   dup = dh act(gate),   dgate = dh up act'(gate).
// From checkpoints gate and up are q * scale in fp32, not rounded to the
// element type in between.
//
// Measured on GB300, GPU time of a call in a CUDA graph over tensors that take
// turns, over 600 MB of them, so that nothing is left in L2; in parentheses the
// time of the bytes, a checkpoint's scales among them, at the 6786 GB/s of a copy
// (what reads more than it writes can be a little faster).  bf16 [4096, 12288],
// silu, gate and up side by side: forward 46.2 us (44.5), with both checkpoints
// 66.1 (59.8), backward 75.5 (74.2), from checkpoints and with h 77.7 (74.6); fp32
// [4096, 6144] 44.8 (44.5), 53.0 (52.2), 73.5 (74.2), 68.6 (67.0).  bf16 [8192,
// 16384] to 8 bits 67.8 (59.9), back 67.8 (59.9); fp32 101.8 (99.5), 109.2 (99.5).
// The checkpoints' rounding (about 14 instructions an element) and the writes'
// share of the traffic are what is left.

#include "tsx_oct.cuh"

namespace tsx {
namespace {

using namespace dev;

// Rows whose loads a thread issues before it uses the first: of one operand read
// from 8 bits, of two or three, and of one to be packed.  bf16 [16384, 16384]
// packed and unpacked: unpacking 2, 4 or 8 rows at once the same, packing 8 rows
// 266 us, 12 274, 16 296.  Gated: 4 rows took 303.7 us in place of 305.2 for the
// gradient of bf16 [16384, 12288], but 12.5 in place of 11.3 for fp32 [1777,
// 2731], whose octs are no vectors, and 3.7 in place of 2.6 for [256, 1024] (three
// sets of tensors in turn).
constexpr int kRowsAtOnce = 4;
constexpr int kGatedRows = 2;
template <int DT>
TSX_HD constexpr int pack_rows() { return DT == TSX_F32 ? 4 : 8; }

struct Place {
    OctAt at;
    int64_t row0;   // the thread's first row; the others are P apart
    int ch;         // its first channel, counted from the row's start
    int rows;       // how many of its rows exist (0 for spare threads of the last warp)
    int most;       // the most that a thread of the CTA has
    bool live;      // the thread has channels
};

template <bool VEC, int ROWS>
__device__ __forceinline__ Place place(const RowLayout& lay)
{
    Place s;
    const int p = lane_of(threadIdx.x, lay.per_v), v = static_cast<int>(threadIdx.x) - p * lay.V;
    const int chunk0 = static_cast<int>(blockIdx.y) * lay.chunk_cols;
    const int cols = min(lay.chunk_cols, lay.cols - chunk0);
    s.at = oct_at<VEC>(v, lay.team, cols);
    s.ch = chunk0 + s.at.ch;
    s.live = p < lay.P && s.at.ch < cols;
    const uint32_t first = blockIdx.x * (lay.P * ROWS);   // rows < 2^31
    s.row0 = first + p;
    // rows that the CTA has: ROWS * P, or fewer at the end
    const int left = static_cast<int>(min(static_cast<uint32_t>(lay.rows) - first, static_cast<uint32_t>(lay.P * ROWS)));
    s.rows = s.most = 0;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        s.rows += p < lay.P && left > i * lay.P + p ? 1 : 0;
        s.most += left > i * lay.P ? 1 : 0;
    }
    return s;
}

// N rows of an operand; those that do not exist are zeros.
template <int DT, bool VEC, int N>
__device__ __forceinline__ void load_rows(const Place& s, const void* base, int64_t pitch, int P, Oct<DT> (&o)[N])
{
    const char* p = oct_ptr<DT>(base, s.row0, pitch, s.ch);
    const int64_t step = P * pitch * elem_size(DT);
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (s.live && i < s.rows)
            o[i] = oct_load<DT, VEC>(p + i * step, s.at);
        else
            oct_zero(o[i]);
}

// The same of a checkpoint's numbers and scales.
template <bool VEC, int N>
__device__ __forceinline__ void load_held(const Place& s, const void* q, const float* scale, const RowLayout& lay,
                                          int64_t blocks, int block, Held (&h)[N], float (&sc)[N])
{
    const uint8_t* p = static_cast<const uint8_t*>(q) + s.row0 * lay.cols + s.ch;
    const float* ps = scale + s.row0 * blocks + block_of(s.ch, block);
    const int64_t step = static_cast<int64_t>(lay.P) * lay.cols, step_s = lay.P * blocks;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (s.live && i < s.rows) {
            h[i] = held_load<VEC>(p + i * step, s.at);
            sc[i] = __ldg(ps + i * step_s);
        }
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kLayerThreads) pack_kernel(PackArgs a, const void* x, HeldOut held)
{
    constexpr int N = pack_rows<DT>();
    const Place s = place<VEC, N>(a.lay);
    Oct<DT> o[N];
    load_rows<DT, VEC>(s, x, a.pitch, a.lay.P, o);
    HeldPtr to(held, s.row0, a.lay.P, a.lay.cols, a.blocks, s.ch, a.block);
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const Oct<DT> four[4] = {o[i], o[i + 1], o[i + 2], o[i + 3]};
        if (i < s.most)
            hold_rows<DT, VEC>(four, s.live, s.at, a.lay.team, a.form, HeldRows{to, s.rows - i});
        to.advance(4);
    }
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kLayerThreads) unpack_kernel(PackArgs a, const void* q, const float* scale, void* x)
{
    const Place s = place<VEC, kRowsAtOnce>(a.lay);
    Held h[kRowsAtOnce];
    float sc[kRowsAtOnce];
    load_held<VEC>(s, q, scale, a.lay, a.blocks, a.block, h, sc);
    char* p = oct_ptr<DT>(x, s.row0, a.pitch, s.ch);
    const int64_t step = a.lay.P * a.pitch * elem_size(DT);
#pragma unroll
    for (int i = 0; i < kRowsAtOnce; ++i)
        if (s.live && i < s.rows) {
            float2 f[4];
            held_floats(h[i], sc[i], a.form, f);
            oct_store<DT, VEC>(p + i * step, s.at, oct_round<DT>(f));
        }
}

template <int DT, bool VEC, bool HOLD>
__global__ void __launch_bounds__(kLayerThreads)
    gated_kernel(GatedArgs a, const void* gate, const void* up, void* h, HeldOut held_gate, HeldOut held_up)
{
    const Place s = place<VEC, kGatedRows>(a.lay);
    Oct<DT> g[kGatedRows], u[kGatedRows];
    load_rows<DT, VEC>(s, gate, a.in_pitch, a.lay.P, g);
    load_rows<DT, VEC>(s, up, a.in_pitch, a.lay.P, u);
    char* ph = oct_ptr<DT>(h, s.row0, a.out_pitch, s.ch);
    const int64_t step = a.lay.P * a.out_pitch * elem_size(DT);
    by_act(a.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < kGatedRows; ++i) {
            float2 fg[4], fu[4], fh[4];
            oct_floats(g[i], fg);
            oct_floats(u[i], fu);
            act_value(act, fg, fh);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                fh[j] = __fmul2_rn(fh[j], fu[j]);
            if (s.live && i < s.rows)
                oct_store<DT, VEC>(ph + i * step, s.at, oct_round<DT>(fh));
        }
    });
    if constexpr (HOLD) {
        static_assert(kGatedRows == 2, "four octs");
        const Oct<DT> four[4] = {g[0], g[1], u[0], u[1]};
        hold_rows<DT, VEC>(four, s.live, s.at, a.lay.team, a.form,
                           HeldPairs{HeldPtr(held_gate, s.row0, a.lay.P, a.lay.cols, a.blocks, s.ch, a.block),
                                     HeldPtr(held_up, s.row0, a.lay.P, a.lay.cols, a.blocks, s.ch, a.block), s.rows});
    }
}

template <int DT, bool VEC, bool HELD>
__global__ void __launch_bounds__(kLayerThreads)
    gated_backward_kernel(GatedArgs a, const void* dh, Saved gate, Saved up, void* dgate, void* dup, void* h)
{
    const Place s = place<VEC, kGatedRows>(a.lay);
    Oct<DT> d[kGatedRows], g[kGatedRows], u[kGatedRows];
    Held qg[kGatedRows], qu[kGatedRows];
    float sg[kGatedRows], su[kGatedRows];
    load_rows<DT, VEC>(s, dh, a.out_pitch, a.lay.P, d);
    if constexpr (HELD) {
        load_held<VEC>(s, gate.q, gate.scale, a.lay, a.blocks, a.block, qg, sg);
        load_held<VEC>(s, up.q, up.scale, a.lay, a.blocks, a.block, qu, su);
    } else {
        load_rows<DT, VEC>(s, gate.x, a.in_pitch, a.lay.P, g);
        load_rows<DT, VEC>(s, up.x, a.in_pitch, a.lay.P, u);
    }
    char* pg = oct_ptr<DT>(dgate, s.row0, a.in_pitch, s.ch);
    char* pu = oct_ptr<DT>(dup, s.row0, a.in_pitch, s.ch);
    char* ph = oct_ptr<DT>(h, s.row0, a.out_pitch, s.ch);
    const int64_t in_step = a.lay.P * a.in_pitch * elem_size(DT), out_step = a.lay.P * a.out_pitch * elem_size(DT);
#pragma unroll
    for (int i = 0; i < kGatedRows; ++i) {
        if (!(s.live && i < s.rows))
            continue;
        float2 fd[4], fg[4], fu[4];
        oct_floats(d[i], fd);
        if constexpr (HELD) {
            held_floats(qg[i], sg[i], a.form, fg);
            held_floats(qu[i], su[i], a.form, fu);
        } else {
            oct_floats(g[i], fg);
            oct_floats(u[i], fu);
        }
        float2 og[4], ou[4], oh[4], value[4], slope[4];
        act_both(a.act, fg, value, slope);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            og[j] = __fmul2_rn(__fmul2_rn(fd[j], fu[j]), slope[j]);
            ou[j] = __fmul2_rn(fd[j], value[j]);
            oh[j] = __fmul2_rn(value[j], fu[j]);
        }
        oct_store<DT, VEC>(pg + i * in_step, s.at, oct_round<DT>(og));
        oct_store<DT, VEC>(pu + i * in_step, s.at, oct_round<DT>(ou));
        if (h)
            oct_store<DT, VEC>(ph + i * out_step, s.at, oct_round<DT>(oh));
    }
}

dim3 grid_of(const RowLayout& lay, int rows_at_once)
{
    const int64_t per = int64_t(lay.P) * rows_at_once;
    return dim3(unsigned((lay.rows + per - 1) / per), unsigned(lay.chunks));
}

}  // namespace

// f<DT, VEC>(...) for the runtime dtype and vec.
#define TSX_BY_TYPE(dtype, vec, CALL)                                        \
    do {                                                                     \
        if (vec) {                                                           \
            if ((dtype) == TSX_F16) { CALL(TSX_F16, true); }                 \
            else if ((dtype) == TSX_BF16) { CALL(TSX_BF16, true); }          \
            else { CALL(TSX_F32, true); }                                    \
        } else {                                                             \
            if ((dtype) == TSX_F16) { CALL(TSX_F16, false); }                \
            else if ((dtype) == TSX_BF16) { CALL(TSX_BF16, false); }         \
            else { CALL(TSX_F32, false); }                                   \
        }                                                                    \
    } while (0)

cudaError_t launch_pack(int dtype, const PackArgs& a, const void* x, HeldOut held, cudaStream_t st)
{
    const dim3 grid = grid_of(a.lay, dtype == TSX_F32 ? pack_rows<TSX_F32>() : pack_rows<TSX_BF16>());
    cudaError_t e = cudaSuccess;
#define CALL(DT, VEC) e = launch_grid<pack_kernel<DT, VEC>>(grid, a.lay.threads, 0, 1, false, st, a, x, held)
    TSX_BY_TYPE(dtype, a.lay.vec, CALL);
#undef CALL
    return e;
}

cudaError_t launch_unpack(int dtype, const PackArgs& a, const void* q, const float* scale, void* x, cudaStream_t st)
{
    const dim3 grid = grid_of(a.lay, kRowsAtOnce);
    cudaError_t e = cudaSuccess;
#define CALL(DT, VEC) e = launch_grid<unpack_kernel<DT, VEC>>(grid, a.lay.threads, 0, 1, false, st, a, q, scale, x)
    TSX_BY_TYPE(dtype, a.lay.vec, CALL);
#undef CALL
    return e;
}

cudaError_t launch_gated(int dtype, const GatedArgs& a, const void* gate, const void* up, void* h, HeldOut held_gate,
                         HeldOut held_up, cudaStream_t st)
{
    const dim3 grid = grid_of(a.lay, kGatedRows);
    cudaError_t e = cudaSuccess;
#define CALL(DT, VEC)                                                                                                   \
    e = held_gate.q ? launch_grid<gated_kernel<DT, VEC, true>>(grid, a.lay.threads, 0, 1, false, st, a, gate, up, h,    \
                                                               held_gate, held_up)                                     \
                    : launch_grid<gated_kernel<DT, VEC, false>>(grid, a.lay.threads, 0, 1, false, st, a, gate, up, h,   \
                                                                held_gate, held_up)
    TSX_BY_TYPE(dtype, a.lay.vec, CALL);
#undef CALL
    return e;
}

cudaError_t launch_gated_backward(int dtype, const GatedArgs& a, const void* dh, Saved gate, Saved up, void* dgate,
                                  void* dup, void* h, cudaStream_t st)
{
    const dim3 grid = grid_of(a.lay, kGatedRows);
    cudaError_t e = cudaSuccess;
#define CALL(DT, VEC)                                                                                               \
    e = gate.q ? launch_grid<gated_backward_kernel<DT, VEC, true>>(grid, a.lay.threads, 0, 1, false, st, a, dh,     \
                                                                   gate, up, dgate, dup, h)                         \
               : launch_grid<gated_backward_kernel<DT, VEC, false>>(grid, a.lay.threads, 0, 1, false, st, a, dh,    \
                                                                    gate, up, dgate, dup, h)
    TSX_BY_TYPE(dtype, a.lay.vec, CALL);
#undef CALL
    return e;
}

}  // namespace tsx
