// score.cu -- log probabilities of given tokens, with rank, entropy and the best alternatives, in one
// pass over the logits. With x = logits of a row and R a reference,
//     s = sum 2^(x log2 e - R),  t = sum (x log2 e - R) 2^(x log2 e - R),
//     lse = (R + log2 s) ln 2,   entropy = ln s - ln 2 * t / s,
// both kept relative to each lane's own running reference and moved by 2^(R - R') when that grows
// (t also by s (R - R')). The rank counts the tokens in front of the given one on the way; the best
// tokens are collected as in beam.cu.
//
// The bytes of the logits bound it (the floor). A CTA has a row, or the splits of a row one each
// where there are few, of which the last to finish joins them.
#include "vocab.cuh"

namespace sfi {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
// -150 is below every power that 32 bits hold: a term of it adds nothing, and 0 * -inf does not arise
constexpr float kNothing = -150.f;

// Sums of a set of tokens relative to their reference (in units of 2^4, see vocab.cuh).
struct Sums {
    float R, s, t;
    int front;
};

// a and b relative to the larger reference; a sum that is not a number stays one.
template <bool ENT>
__device__ __forceinline__ Sums join(const Sums &a, const Sums &b)
{
    Sums o;
    o.R = fmaxf(a.R, b.R);
    o.front = a.front + b.front;
    o.s = o.t = 0.f;
    const Sums *in[2] = {&a, &b};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const Sums &v = *in[i];
        if (v.s != 0.f) {
            const float d = o.R > -CUDART_INF_F ? 4.f * (v.R - o.R) : 0.f;
            const float w = ex2(d);
            o.s += v.s * w;
            if (ENT && w != 0.f)
                o.t += (v.t + v.s * d) * w;
        }
    }
    return o;
}

template <typename T, bool TOP, bool RANK, bool ENT>
__global__ void __launch_bounds__(kScoreThreads, 4) score_kernel(const ScoreParams p)
{
    // candidates that wait to be inserted, in any order: fewer than 32 and a chunk's
    __shared__ float cand_x[TOP ? kScoreWarps : 1][TOP ? 32 * kLaneTok + 32 : 1];
    __shared__ int cand_v[TOP ? kScoreWarps : 1][TOP ? 32 * kLaneTok + 32 : 1], n_cand[kScoreWarps];
    __shared__ float sh_x[TOP ? kMaxTop : 1][kScoreWarps];
    __shared__ int sh_v[TOP ? kMaxTop : 1][kScoreWarps];
    __shared__ volatile int top[kScoreWarps];        // (as order())
    __shared__ Sums sh_sums[kScoreWarps];
    __shared__ int sh_last;
    constexpr int V = Chunk<T>::kV;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = p.n_top;
    const int row = p.splits == 1 ? blockIdx.x : blockIdx.x / p.splits;
    const int split = p.splits == 1 ? 0 : blockIdx.x - row * p.splits;
    if (TOP && tid < kScoreWarps) {
        top[tid] = order(-CUDART_INF_F);
        n_cand[tid] = 0;
    }
    pdl_trigger();
    pdl_wait();
    const T *x0 = static_cast<const T *>(p.logits) + static_cast<size_t>(row) * p.row_stride;
    const int given = p.token ? p.token[row] : -1;
    const bool has = given >= 0 && given < p.vocab;
    const float xg = has ? static_cast<float>(x0[given]) : CUDART_NAN_F;
    if (TOP)
        __syncthreads();
    const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(x0) & 15u) / sizeof(T));
    const int pieces = (p.vocab + shift + V - 1) / V;
    constexpr int kStep = 32 * (kLaneTok / V);               // pieces per chunk
    Best best;
    best.clear();
    bool fresh = true;          // (the same in every lane, as is all that decides a branch here)
    int mine = order(-CUDART_INF_F);    // the warp's highest logit
    // the candidates that wait go into the list, without those that the CTA's bound has passed
    auto insert_waiting = [&] {
        __syncwarp();
        const int n = n_cand[warp];
        const float floor = unorder(__reduce_min_sync(kAll, top[lane & (kScoreWarps - 1)]));
        for (int i = 0; i < n; i += 32) {
            const float cx = i + lane < n ? cand_x[warp][i + lane] : -CUDART_INF_F;
            best.offer(cx, i + lane < n && cx >= floor ? cand_v[warp][i + lane] : -1, K, lane);
        }
        __syncwarp();
        if (lane == 0)
            n_cand[warp] = 0;
        if (K > kScoreWarps && lane == (K - 1) / kScoreWarps)
            top[warp] = order(best.x);
        __syncwarp();
    };
    Sums a = {-CUDART_INF_F, 0.f, 0.f, 0};
    int c = (split * kScoreWarps + warp) * kStep;
    const int stride = p.splits * kScoreWarps * kStep;
    uint4 w[kLaneTok / V];
    if (c < pieces)
        load_chunk(x0, shift, p.vocab, c, lane, w);
    for (; c < pieces; c += stride) {
        float x[kLaneTok];
#pragma unroll
        for (int i = 0; i < kLaneTok / V; ++i)
            Chunk<T>::unpack(w[i], x + V * i);
        if (c + stride < pieces)
            load_chunk(x0, shift, p.vocab, c + stride, lane, w);
        const int v0 = (c + lane) * V - shift;
        // (tokens grow with j, so the first of equal logits is the lowest token)
        auto token = [&](int j) { return v0 + 32 * V * (j / V) + j % V; };
        float cm = -CUDART_INF_F;       // (fmaxf drops NaN)
#pragma unroll
        for (int j = 0; j < kLaneTok; ++j)
            cm = fmaxf(cm, x[j]);
        const float rn = fmaxf(a.R, cm * kLog2e4);
        if (fabsf(rn) < kLarge * kLog2e4) {
            if (a.s != 0.f) {
                const float d = 4.f * (a.R - rn), f = ex2(d);
                if (ENT)
                    a.t = (a.t + a.s * d) * f;
                a.s *= f;
                if (ENT && f == 0.f)
                    a.t = 0.f;          // (d may be beyond what 32 bits hold)
            }
            a.R = rn;
            const uint64_t c2 = pack2(kLog2e, kLog2e), r2 = pack2(-4.f * rn, -4.f * rn);
            uint64_t acc = 0, ent = 0;
#pragma unroll
            for (int j = 0; j < kLaneTok; j += 2) {
                float2 z = unpack2(fma2(pack2(x[j], x[j + 1]), c2, r2));
                const uint64_t e = pack2(ex2(z.x), ex2(z.y));
                acc = add2(acc, e);
                if (ENT)
                    ent = fma2(e, pack2(fmaxf(z.x, kNothing), fmaxf(z.y, kNothing)), ent);
            }
            const float2 s2 = unpack2(acc);
            a.s += s2.x + s2.y;
            if (ENT) {
                const float2 t2 = unpack2(ent);
                a.t += t2.x + t2.y;
            }
        } else {
            // a largest logit from kLarge on, of either sign, or -inf alone, or NaN or +inf, which
            // have to show in the sum
            const float rm = cm > -CUDART_INF_F ? fmaxf(a.R, reference(cm)) : a.R;
            if (a.s != 0.f && rm > a.R) {
                const float d = 4.f * (a.R - rm), f = ex2(d);
                a.t = ENT && f != 0.f ? (a.t + a.s * d) * f : 0.f;
                a.s *= f;
            }
            a.R = rm;
#pragma unroll
            for (int j = 0; j < kLaneTok; ++j) {
                const float z = 4.f * (reference(x[j]) - rm), e = ex2(z);
                a.s += x[j] > -CUDART_INF_F ? e : x[j] == x[j] ? 0.f : CUDART_NAN_F;
                if (ENT && e != 0.f && x[j] > -CUDART_INF_F)
                    a.t += e * z;
            }
        }
        if (RANK) {
#pragma unroll
            for (int j = 0; j < kLaneTok; ++j) {
                // (what lies beyond the row's ends is -inf, and may be equal to the token's)
                const int v = token(j);
                a.front += x[j] > xg || (x[j] == xg && v < given && v >= 0) ? 1 : 0;
            }
        }
        if (TOP) {
            // Tokens that beat the K-th best so far; see beam.cu.
            const float floor = unorder(__reduce_min_sync(kAll, top[lane & (kScoreWarps - 1)]));
            if (__any_sync(kAll, cm >= floor && (cm > best.tx || best.tv < 0))) {
                if (K <= kScoreWarps) {
                    mine = max(mine, __reduce_max_sync(kAll, order(cm)));
                    if (lane == 0)
                        top[warp] = mine;
                }
                int taken = -1;
                if (fresh) {
                    float cx = -CUDART_INF_F;
#pragma unroll
                    for (int j = kLaneTok - 1; j >= 0; --j) {
                        if (x[j] >= cx && token(j) >= 0 && token(j) < p.vocab) {
                            cx = x[j];
                            taken = token(j);
                        }
                    }
                    best.start(cx, taken, K, lane);
                }
                const float least = fmaxf(floor, best.tx);
#pragma unroll
                for (int j = 0; j < kLaneTok; ++j) {
                    if (x[j] >= least) {
                        const int v = token(j);
                        if (v != taken && v >= 0 && v < p.vocab) {
                            const int at = atomicAdd(&n_cand[warp], 1);
                            cand_x[warp][at] = x[j];
                            cand_v[warp][at] = v;
                        }
                    }
                }
                __syncwarp();
                if (fresh || n_cand[warp] >= 32)
                    insert_waiting();
                fresh = false;
            }
        }
    }
    if (TOP)
        insert_waiting();
    // the warp's sums
    auto warp_join = [&](Sums v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            Sums b;
            b.R = __shfl_xor_sync(kAll, v.R, o);
            b.s = __shfl_xor_sync(kAll, v.s, o);
            b.t = ENT ? __shfl_xor_sync(kAll, v.t, o) : 0.f;
            b.front = RANK ? __shfl_xor_sync(kAll, v.front, o) : 0;
            v = join<ENT>(v, b);
        }
        return v;
    };
    a = warp_join(a);
    if (lane == 0)
        sh_sums[warp] = a;
    if (TOP && lane < K) {
        sh_x[lane][warp] = best.x;
        sh_v[lane][warp] = best.v;
    }
    __syncthreads();
    const Sums none = {-CUDART_INF_F, 0.f, 0.f, 0};
    if (warp == 0) {
        a = warp_join(lane < kScoreWarps ? sh_sums[lane] : none);
        if (TOP) {
            // all warps' j-th before any (j + 1)-th, so that the first 32 settle most
            best.clear();
            best.start((&sh_x[0][0])[lane], lane < K * kScoreWarps ? (&sh_v[0][0])[lane] : -1, K, lane);
            for (int i = 32; i < K * kScoreWarps; i += 32)
                best.offer((&sh_x[0][0])[min(i + lane, K * kScoreWarps - 1)],
                           i + lane < K * kScoreWarps ? (&sh_v[0][0])[i + lane] : -1, K, lane);
        }
    }
    if (p.splits > 1) {
        if (warp == 0) {
            const size_t part = static_cast<size_t>(row) * p.splits + split;
            if (lane == 0)
                p.part[part] = make_float4(a.R, a.s, a.t, __int_as_float(a.front));
            if (TOP && lane < K) {
                const size_t at = (static_cast<size_t>(row) * K + lane) * p.splits + split;
                p.part_x[at] = best.x;
                p.part_v[at] = best.v;
            }
            __threadfence();
        }
        __syncthreads();
        if (tid == 0)
            sh_last = atomic_add_acq_rel_gpu(p.tickets + row, 1) == p.splits - 1;
        __syncthreads();
        if (!sh_last || warp != 0)
            return;
        __threadfence();
        if (lane == 0)
            p.tickets[row] = 0;
        const size_t part = static_cast<size_t>(row) * p.splits;
        a = none;
        for (int i = lane; i < p.splits; i += 32) {
            const float4 v = __ldcg(p.part + part + i);
            a = join<ENT>(a, Sums{v.x, v.y, v.z, __float_as_int(v.w)});
        }
        a = warp_join(a);
        if (TOP) {
            best.clear();
            const int n = K * p.splits;
            for (int i = 0; i < n; i += 32) {
                const float ox = i + lane < n ? __ldcg(p.part_x + part * K + i + lane) : 0.f;
                const int ov = i + lane < n ? __ldcg(p.part_v + part * K + i + lane) : -1;
                if (i == 0)
                    best.start(ox, ov, K, lane);
                else
                    best.offer(ox, ov, K, lane);
            }
        }
    }
    if (warp != 0)
        return;
    const float ls = logf(a.s);
    const bool sound = isfinite(a.R) && isfinite(ls);
    // lse less ln s, in double: in fp32 it would round at the size of the logits. From kLarge on
    // the reference is half the largest logit.
    const double ref = fabsf(a.R) < kLarge * kLog2e4 ? a.R / static_cast<double>(kLog2e4) : 2. * a.R;
    // (a probability is at most 1 and entropy at least 0, whatever the roundings say)
    auto log_p = [&](float x) { return sound ? fminf(static_cast<float>(x - ref - ls), 0.f) : CUDART_NAN_F; };
    if (lane == 0) {
        if (p.logprob)
            p.logprob[row] = given < 0 ? 0.f : has ? log_p(xg) : CUDART_NAN_F;
        if (RANK)
            p.rank[row] = has && sound ? a.front : -1;
        if (ENT)
            p.entropy[row] = sound ? fmaxf(ls - a.t / a.s * CUDART_LN2_F, 0.f) : CUDART_NAN_F;
    }
    if (TOP && lane < K) {
        const size_t at = static_cast<size_t>(row) * K + lane;
        p.top_token[at] = sound ? best.v : -1;
        p.top_logprob[at] = log_p(best.x);
    }
}

template <typename T, bool TOP>
cudaError_t launch_top(const ScoreParams &p, cudaStream_t stream)
{
    const dim3 grid(p.n_rows * p.splits), block(kScoreThreads);
    if (p.rank)
        return p.entropy ? launch_pdl(score_kernel<T, TOP, true, true>, grid, block, 0, stream, p)
                         : launch_pdl(score_kernel<T, TOP, true, false>, grid, block, 0, stream, p);
    return p.entropy ? launch_pdl(score_kernel<T, TOP, false, true>, grid, block, 0, stream, p)
                     : launch_pdl(score_kernel<T, TOP, false, false>, grid, block, 0, stream, p);
}

template <typename T>
cudaError_t launch_type(const ScoreParams &p, cudaStream_t stream)
{
    return p.n_top > 0 ? launch_top<T, true>(p, stream) : launch_top<T, false>(p, stream);
}

}  // namespace

cudaError_t launch_score(const ScoreParams &p, cudaStream_t stream)
{
    const cudaError_t e = p.logits_fp32 ? launch_type<float>(p, stream) : launch_type<__nv_bfloat16>(p, stream);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sfi
