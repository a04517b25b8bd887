// beam.cu -- beam search's selection: one pass over the logits of every row for the softmax's
// maximum and sum and the row's best tokens, then the best n_beams of each group.
//
// Within a row s(r, v) = cum + x[v] - lse is monotone in x, so a row's n_beams best tokens by
// logit are all that its group can need: every CTA reduces a slice of a row to (max, sum, best
// tokens), and the last CTA of a group joins its rows' slices.
#include "sfi_device.cuh"

#include <math_constants.h>

namespace sfi {
namespace {

constexpr int kBeamThreads = 256;

// a before b: higher logit, then lower token (empty places, v < 0, last)
__device__ __forceinline__ bool better(float xa, int va, float xb, int vb)
{
    if (va < 0 || vb < 0)
        return va >= 0;
    return xa > xb || (xa == xb && va < vb);
}

struct Cand {
    float key, x, s;
    int row, v;
};

__device__ __forceinline__ bool better(const Cand &a, const Cand &b)
{
    if (a.v < 0 || b.v < 0)
        return a.v >= 0;
    if (a.key != b.key)
        return a.key > b.key;
    if (a.row != b.row)
        return a.row < b.row;
    return a.x > b.x || (a.x == b.x && a.v < b.v);
}

template <int KT>
__global__ void __launch_bounds__(kBeamThreads) beam_kernel(const BeamParams p)
{
    __shared__ float sh_m[8], sh_s[8], sh_x[8];
    __shared__ int sh_v[8], sh_t[8];
    __shared__ Cand sh_c[8];
    __shared__ int sh_win, sh_last;
    __shared__ float row_max[kMaxBeams], row_log[kMaxBeams], row_cum[kMaxBeams], row_scale[kMaxBeams];
    __shared__ int row_kind[kMaxBeams];   // 0 live, 1 finished, 2 all scores -inf
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = p.n_beams, row = blockIdx.y, split = blockIdx.x;
    pdl_wait();
    if (!(p.done && p.done[row])) {
        const int per = (p.vocab + p.splits - 1) / p.splits;
        const int v0 = split * per, v1 = min(p.vocab, v0 + per);
        float m = -CUDART_INF_F, s = 0.f, bx[KT];
        int bv[KT];
#pragma unroll
        for (int j = 0; j < KT; ++j) {
            bx[j] = -CUDART_INF_F;
            bv[j] = -1;
        }
        bool nan = false;
        for (int v = v0 + tid; v < v1; v += kBeamThreads) {
            const size_t at = static_cast<size_t>(row) * p.row_stride + v;
            float x = p.logits_fp32 ? static_cast<const float *>(p.logits)[at]
                                    : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.logits)[at]);
            nan = nan || x != x;
            if (x > m) {
                s = s * expf(m - x) + 1.f;
                m = x;
            } else if (m > -CUDART_INF_F) {
                s += expf(x - m);
            }
            if (better(x, v, bx[KT - 1], bv[KT - 1])) {
                int w = v;
#pragma unroll
                for (int j = 0; j < KT; ++j) {
                    if (better(x, w, bx[j], bv[j])) {
                        const float tx = bx[j];
                        const int tv = bv[j];
                        bx[j] = x;
                        bv[j] = w;
                        x = tx;
                        w = tv;
                    }
                }
            }
        }
        if (nan)
            s = CUDART_NAN_F;
        // maximum and sum of the slice
        float bm = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
        if (lane == 0)
            sh_m[warp] = bm;
        __syncthreads();
        bm = sh_m[0];
        for (int w = 1; w < 8; ++w)
            bm = fmaxf(bm, sh_m[w]);
        // (a sum without a finite maximum is 0, or NaN; inf - inf gives the NaN wanted)
        float bs = s == 0.f ? 0.f : s * expf(m - bm);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            bs += __shfl_xor_sync(0xffffffffu, bs, o);
        if (lane == 0)
            sh_s[warp] = bs;
        __syncthreads();
        const size_t part = static_cast<size_t>(row) * p.splits + split;
        if (tid == 0) {
            bs = 0.f;
            for (int w = 0; w < 8; ++w)
                bs += sh_s[w];
            p.part_stat[part] = make_float2(bm, bs);
        }
        // K rounds: the best head of all threads' lists
        for (int k = 0; k < K; ++k) {
            float x = bx[0];
            int v = bv[0], t = tid;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float ox = __shfl_xor_sync(0xffffffffu, x, o);
                const int ov = __shfl_xor_sync(0xffffffffu, v, o), ot = __shfl_xor_sync(0xffffffffu, t, o);
                if (better(ox, ov, x, v)) {
                    x = ox;
                    v = ov;
                    t = ot;
                }
            }
            if (lane == 0) {
                sh_x[warp] = x;
                sh_v[warp] = v;
                sh_t[warp] = t;
            }
            __syncthreads();
            if (tid == 0) {
                int best = 0;
                for (int w = 1; w < 8; ++w)
                    if (better(sh_x[w], sh_v[w], sh_x[best], sh_v[best]))
                        best = w;
                p.part_x[part * K + k] = sh_x[best];
                p.part_v[part * K + k] = sh_v[best];
                sh_win = sh_v[best] >= 0 ? sh_t[best] : -1;
            }
            __syncthreads();
            if (tid == sh_win) {
#pragma unroll
                for (int j = 0; j + 1 < KT; ++j) {
                    bx[j] = bx[j + 1];
                    bv[j] = bv[j + 1];
                }
                bv[KT - 1] = -1;
            }
        }
    }
    // the last CTA of the group joins
    const int group = row / K;
    __syncthreads();
    if (tid == 0)
        sh_last = atomic_add_acq_rel_gpu(p.tickets + group, 1) == K * p.splits - 1;
    __syncthreads();
    if (!sh_last)
        return;
    if (tid == 0)
        p.tickets[group] = 0;
    if (tid < K) {
        const int r = group * K + tid;
        const float cum = p.cum[r];
        int kind = 0;
        float m = -CUDART_INF_F, ls = 0.f;
        if (p.done && p.done[r]) {
            kind = 1;
        } else {
            float s = 0.f;
            for (int i = 0; i < p.splits; ++i) {
                const float2 st = __ldcg(p.part_stat + static_cast<size_t>(r) * p.splits + i);
                m = fmaxf(m, st.x);
            }
            for (int i = 0; i < p.splits; ++i) {
                const float2 st = __ldcg(p.part_stat + static_cast<size_t>(r) * p.splits + i);
                s += st.y == 0.f ? 0.f : st.y * expf(st.x - m);
            }
            ls = logf(s);   // kept apart from the maximum: their sum would round at |m|
            if (!isfinite(m) || !isfinite(ls) || !isfinite(cum))
                kind = 2;
        }
        row_kind[tid] = kind;
        row_max[tid] = m;
        row_log[tid] = ls;
        row_cum[tid] = cum;
        row_scale[tid] = p.rank_scale ? p.rank_scale[r] : 1.f;
    }
    __syncthreads();
    Cand last;
    last.v = -2;
    for (int k = 0; k < K; ++k) {
        Cand best;
        best.v = -1;
        best.key = best.x = best.s = 0.f;
        best.row = 0;
        const int each = p.splits * K;
        for (int i = tid; i < K * each; i += kBeamThreads) {
            Cand c;
            c.row = i / each;
            const int j = i - c.row * each, kind = row_kind[c.row];
            if (kind == 0) {
                const size_t at = static_cast<size_t>(group * K + c.row) * each + j;
                c.x = __ldcg(p.part_x + at);
                c.v = __ldcg(p.part_v + at);
                c.s = row_cum[c.row] + ((c.x - row_max[c.row]) - row_log[c.row]);
            } else if (kind == 1) {
                c.v = j == 0 ? p.eos : -1;
                c.x = 0.f;
                c.s = isfinite(row_cum[c.row]) ? row_cum[c.row] : -CUDART_INF_F;
            } else {
                c.v = j < p.vocab && j < K ? j : -1;
                c.x = 0.f;
                c.s = -CUDART_INF_F;
            }
            c.key = c.s * row_scale[c.row];
            // after the one chosen before it, and ahead of the best so far
            if (c.v >= 0 && (last.v == -2 || better(last, c)) && better(c, best))
                best = c;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            Cand c;
            c.key = __shfl_xor_sync(0xffffffffu, best.key, o);
            c.x = __shfl_xor_sync(0xffffffffu, best.x, o);
            c.s = __shfl_xor_sync(0xffffffffu, best.s, o);
            c.row = __shfl_xor_sync(0xffffffffu, best.row, o);
            c.v = __shfl_xor_sync(0xffffffffu, best.v, o);
            if (better(c, best))
                best = c;
        }
        if (lane == 0)
            sh_c[warp] = best;
        __syncthreads();
        best = sh_c[0];
        for (int w = 1; w < 8; ++w)
            if (better(sh_c[w], best))
                best = sh_c[w];
        __syncthreads();
        last = best;
        if (tid == 0) {
            const int o = group * K + k, r = group * K + best.row;
            p.parent[o] = r;
            p.token[o] = best.v;
            p.cum_out[o] = best.s;
            if (p.done_out)
                p.done_out[o] = row_kind[best.row] == 1 || best.v == p.eos ? 1 : 0;
        }
    }
}

}  // namespace

cudaError_t launch_beam_select(const BeamParams &p, cudaStream_t stream)
{
    const dim3 grid(p.splits, p.n_groups * p.n_beams), block(kBeamThreads);
    cudaError_t e;
    if (p.n_beams <= 1)
        e = launch_pdl(beam_kernel<1>, grid, block, 0, stream, p);
    else if (p.n_beams <= 4)
        e = launch_pdl(beam_kernel<4>, grid, block, 0, stream, p);
    else if (p.n_beams <= 8)
        e = launch_pdl(beam_kernel<8>, grid, block, 0, stream, p);
    else
        e = launch_pdl(beam_kernel<16>, grid, block, 0, stream, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sfi
