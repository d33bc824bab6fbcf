// Gated activation h = act(gate) * up and its gradient, and the packing of
// activations into 8 bits and back.
//
// All of them are one pass over their operands with a few to a few dozen
// instructions an element, so HBM bounds them.  A thread keeps its eight
// channels and walks rows; it first issues the loads of kRowsAtOnce rows, so
// that enough bytes are in flight without a ring in shared memory, then
// computes and stores them.  Formulas, with p the sigmoid of the activation:
//   dup = dh act(gate),   dgate = dh up act'(gate).
// From checkpoints gate and up are q * scale in fp32, not rounded to the
// element type in between.

#include "tsx_oct.cuh"

namespace tsx {
namespace {

using namespace dev;

// Rows whose loads a thread issues before it uses the first.
constexpr int kRowsAtOnce = 4;

struct Place {
    OctAt at;
    int64_t row0;   // the thread's first row
    int chunk0;     // the run's first channel
    bool live;      // the thread has channels
};

template <bool VEC>
__device__ __forceinline__ Place place(const RowLayout& lay, int rows_at_once)
{
    Place s;
    const int p = static_cast<int>(threadIdx.x) / lay.V, v = static_cast<int>(threadIdx.x) - p * lay.V;
    s.chunk0 = static_cast<int>(blockIdx.y) * lay.chunk_cols;
    const int cols = min(lay.chunk_cols, lay.cols - s.chunk0);
    s.at = oct_at<VEC>(v, lay.team, cols);
    s.live = p < lay.P && s.at.ch < cols;
    s.row0 = static_cast<int64_t>(blockIdx.x) * (lay.P * rows_at_once) + p;
    return s;
}

// An oct to 8 bits with its team's scale, both stored.  Called by whole
// warps; `live` threads hold channels.
template <bool VEC>
__device__ __forceinline__ void hold(const float2 (&f)[4], bool live, const Place& s, int64_t row, int team, int cols,
                                     int block, int64_t blocks, int form, const HeldOut& out)
{
    const uint32_t m = team_max(live ? oct_amax_bits(f) : 0u, team);
    const HeldScale hs = held_scale(m, form);
    if (!live)
        return;
    held_store<VEC>(out.q, row * cols + s.chunk0, s.at, held_round(f, hs, form));
    const int ch = s.chunk0 + s.at.ch;
    if (ch % block == 0)   // the block's first thread
        out.scale[row * blocks + ch / block] = hs.scale;
}

template <bool VEC>
__device__ __forceinline__ float scale_of(const float* scale, int64_t row, int64_t blocks, const Place& s, int block)
{
    return __ldg(scale + row * blocks + (s.chunk0 + s.at.ch) / block);
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kLayerThreads) pack_kernel(PackArgs a, const void* x, HeldOut held)
{
    const Place s = place<VEC>(a.lay, kRowsAtOnce);
    Oct<DT> o[kRowsAtOnce];
#pragma unroll
    for (int i = 0; i < kRowsAtOnce; ++i) {
        const int64_t r = s.row0 + i * a.lay.P;
        oct_zero(o[i]);
        if (s.live && r < a.lay.rows)
            o[i] = oct_load<DT, VEC>(x, r * a.pitch + s.chunk0, s.at);
    }
#pragma unroll
    for (int i = 0; i < kRowsAtOnce; ++i) {
        const int64_t r = s.row0 + i * a.lay.P;
        float2 f[4];
        oct_floats(o[i], f);
        hold<VEC>(f, s.live && r < a.lay.rows, s, r, a.lay.team, a.lay.cols, a.block, a.blocks, a.form, held);
    }
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kLayerThreads) unpack_kernel(PackArgs a, const void* q, const float* scale, void* x)
{
    const Place s = place<VEC>(a.lay, kRowsAtOnce);
    Held h[kRowsAtOnce];
    float sc[kRowsAtOnce];
#pragma unroll
    for (int i = 0; i < kRowsAtOnce; ++i) {
        const int64_t r = s.row0 + i * a.lay.P;
        if (s.live && r < a.lay.rows) {
            h[i] = held_load<VEC>(q, r * a.lay.cols + s.chunk0, s.at);
            sc[i] = scale_of<VEC>(scale, r, a.blocks, s, a.block);
        }
    }
#pragma unroll
    for (int i = 0; i < kRowsAtOnce; ++i) {
        const int64_t r = s.row0 + i * a.lay.P;
        if (s.live && r < a.lay.rows) {
            float2 f[4];
            held_floats(h[i], sc[i], a.form, f);
            oct_store<DT, VEC>(x, r * a.pitch + s.chunk0, s.at, oct_round<DT>(f));
        }
    }
}

// Two inputs: half as many rows at once.
constexpr int kGatedRows = 2;

template <int DT, bool VEC, bool HOLD>
__global__ void __launch_bounds__(kLayerThreads)
    gated_kernel(GatedArgs a, const void* gate, const void* up, void* h, HeldOut held_gate, HeldOut held_up)
{
    const Place s = place<VEC>(a.lay, kGatedRows);
    Oct<DT> g[kGatedRows], u[kGatedRows];
#pragma unroll
    for (int i = 0; i < kGatedRows; ++i) {
        const int64_t r = s.row0 + i * a.lay.P;
        oct_zero(g[i]);
        oct_zero(u[i]);
        if (s.live && r < a.lay.rows) {
            g[i] = oct_load<DT, VEC>(gate, r * a.in_pitch + s.chunk0, s.at);
            u[i] = oct_load<DT, VEC>(up, r * a.in_pitch + s.chunk0, s.at);
        }
    }
#pragma unroll
    for (int i = 0; i < kGatedRows; ++i) {
        const int64_t r = s.row0 + i * a.lay.P;
        const bool live = s.live && r < a.lay.rows;
        float2 fg[4], fu[4], fh[4];
        oct_floats(g[i], fg);
        oct_floats(u[i], fu);
        act_value(a.act, fg, fh);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            fh[j] = __fmul2_rn(fh[j], fu[j]);
        if (live)
            oct_store<DT, VEC>(h, r * a.out_pitch + s.chunk0, s.at, oct_round<DT>(fh));
        if constexpr (HOLD) {
            hold<VEC>(fg, live, s, r, a.lay.team, a.lay.cols, a.block, a.blocks, a.form, held_gate);
            hold<VEC>(fu, live, s, r, a.lay.team, a.lay.cols, a.block, a.blocks, a.form, held_up);
        }
    }
}

template <int DT, bool VEC, bool HELD>
__global__ void __launch_bounds__(kLayerThreads)
    gated_backward_kernel(GatedArgs a, const void* dh, Saved gate, Saved up, void* dgate, void* dup, void* h)
{
    const Place s = place<VEC>(a.lay, kGatedRows);
    Oct<DT> d[kGatedRows], g[kGatedRows], u[kGatedRows];
    Held qg[kGatedRows], qu[kGatedRows];
    float sg[kGatedRows], su[kGatedRows];
#pragma unroll
    for (int i = 0; i < kGatedRows; ++i) {
        const int64_t r = s.row0 + i * a.lay.P;
        if (s.live && r < a.lay.rows) {
            d[i] = oct_load<DT, VEC>(dh, r * a.out_pitch + s.chunk0, s.at);
            if constexpr (HELD) {
                qg[i] = held_load<VEC>(gate.q, r * a.lay.cols + s.chunk0, s.at);
                qu[i] = held_load<VEC>(up.q, r * a.lay.cols + s.chunk0, s.at);
                sg[i] = scale_of<VEC>(gate.scale, r, a.blocks, s, a.block);
                su[i] = scale_of<VEC>(up.scale, r, a.blocks, s, a.block);
            } else {
                g[i] = oct_load<DT, VEC>(gate.x, r * a.in_pitch + s.chunk0, s.at);
                u[i] = oct_load<DT, VEC>(up.x, r * a.in_pitch + s.chunk0, s.at);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kGatedRows; ++i) {
        const int64_t r = s.row0 + i * a.lay.P;
        if (!(s.live && r < a.lay.rows))
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
        oct_store<DT, VEC>(dgate, r * a.in_pitch + s.chunk0, s.at, oct_round<DT>(og));
        oct_store<DT, VEC>(dup, r * a.in_pitch + s.chunk0, s.at, oct_round<DT>(ou));
        if (h)
            oct_store<DT, VEC>(h, r * a.out_pitch + s.chunk0, s.at, oct_round<DT>(oh));
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
    const dim3 grid = grid_of(a.lay, kRowsAtOnce);
#define CALL(DT, VEC) pack_kernel<DT, VEC><<<grid, a.lay.threads, 0, st>>>(a, x, held)
    TSX_BY_TYPE(dtype, a.lay.vec, CALL);
#undef CALL
    return cudaGetLastError();
}

cudaError_t launch_unpack(int dtype, const PackArgs& a, const void* q, const float* scale, void* x, cudaStream_t st)
{
    const dim3 grid = grid_of(a.lay, kRowsAtOnce);
#define CALL(DT, VEC) unpack_kernel<DT, VEC><<<grid, a.lay.threads, 0, st>>>(a, q, scale, x)
    TSX_BY_TYPE(dtype, a.lay.vec, CALL);
#undef CALL
    return cudaGetLastError();
}

cudaError_t launch_gated(int dtype, const GatedArgs& a, const void* gate, const void* up, void* h, HeldOut held_gate,
                         HeldOut held_up, cudaStream_t st)
{
    const dim3 grid = grid_of(a.lay, kGatedRows);
#define CALL(DT, VEC)                                                                                            \
    if (held_gate.q)                                                                                             \
        gated_kernel<DT, VEC, true><<<grid, a.lay.threads, 0, st>>>(a, gate, up, h, held_gate, held_up);          \
    else                                                                                                         \
        gated_kernel<DT, VEC, false><<<grid, a.lay.threads, 0, st>>>(a, gate, up, h, held_gate, held_up)
    TSX_BY_TYPE(dtype, a.lay.vec, CALL);
#undef CALL
    return cudaGetLastError();
}

cudaError_t launch_gated_backward(int dtype, const GatedArgs& a, const void* dh, Saved gate, Saved up, void* dgate,
                                  void* dup, void* h, cudaStream_t st)
{
    const dim3 grid = grid_of(a.lay, kGatedRows);
#define CALL(DT, VEC)                                                                                            \
    if (gate.q)                                                                                                  \
        gated_backward_kernel<DT, VEC, true><<<grid, a.lay.threads, 0, st>>>(a, dh, gate, up, dgate, dup, h);     \
    else                                                                                                         \
        gated_backward_kernel<DT, VEC, false><<<grid, a.lay.threads, 0, st>>>(a, dh, gate, up, dgate, dup, h)
    TSX_BY_TYPE(dtype, a.lay.vec, CALL);
#undef CALL
    return cudaGetLastError();
}

}  // namespace tsx
