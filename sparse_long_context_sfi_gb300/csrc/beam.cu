// beam.cu -- beam search's selection: one pass over the logits of every row for the softmax's
// maximum and sum and the row's best tokens, then the best n_beams of each group.
//
// Within a row s(r, v) = cum + x[v] - lse is monotone in x, so a row's n_beams best tokens by
// logit are all that its group can need. The logits are read once (the floor: their bytes);
// every warp takes 512-token chunks of its row, 16 tokens per lane in registers, the next
// chunk's loads in flight. The best tokens so far lie sorted in the warp's lanes, and a chunk
// whose maximum is below the last of them, or below a bound that the CTA's warps share, costs a
// comparison per lane; tokens that may enter the list wait in shared memory and are inserted
// together, from the last one, so that neither ascending nor descending logits insert every
// token. Warps of a CTA, the CTAs of a row (splits) and the rows of a group are
// joined by the same insertion; the last CTA of a group does the last two.
//
// Issue slots bound it (a token's share at the copy rate is ~22 of fp32, ~11 of bf16), so the
// sums are kept relative to R = fl(max * log2 e): exp(x) / 2^R = 2^(x log2 e - R) is then one
// exact-product multiply-add and an exponential per token, for logits up to 2^29 (beyond: see
// reference()), and only the scores of the chosen few are formed from R, in double.
//
// 256 rows of 128001 fp32 logits: 31.3 us, 4.2 TB/s (floor 19 us). Without any list it takes
// 21.6 us, with the first chunk's alone 26; the rest is tests, waiting tokens and insertions. (304
// rows, which fill the GPU, take no longer than 256, whose 512 CTAs leave some SMs a quarter idle.)
// 4 rows of 32000 bf16: 8.5 us, launch and round trips.
#include "vocab.cuh"

namespace sfi {
namespace {

constexpr int kBeamThreads = 256;
constexpr int kBeamWarps = kBeamThreads / 32;

template <typename T>
__global__ void __launch_bounds__(kBeamThreads, 4) beam_kernel(const BeamParams p)
{
    __shared__ float sh_x[kMaxBeams][kBeamWarps], sh_m[kBeamWarps], sh_s[kBeamWarps];
    __shared__ int sh_v[kMaxBeams][kBeamWarps];
    // candidates that wait to be inserted, in any order: fewer than 32 and a chunk's
    __shared__ float cand_x[kBeamWarps][32 * kLaneTok + 32];
    __shared__ int cand_v[kBeamWarps][32 * kLaneTok + 32], n_cand[kBeamWarps];
    __shared__ volatile int top[kBeamWarps];        // (as order())
    __shared__ float row_x[kMaxBeams][kMaxBeams], row_s[kMaxBeams][kMaxBeams];
    __shared__ int row_v[kMaxBeams][kMaxBeams];
    __shared__ uint8_t row_done[kMaxBeams];
    __shared__ int sh_last;
    constexpr int V = Chunk<T>::kV;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = p.n_beams, row = blockIdx.y, split = blockIdx.x, group = row / K;
    if (tid < kBeamWarps) {
        top[tid] = order(-CUDART_INF_F);
        n_cand[tid] = 0;
    }
    pdl_wait();
    __syncthreads();
    if (!(p.done && p.done[row])) {
        const T *x0 = static_cast<const T *>(p.logits) + static_cast<size_t>(row) * p.row_stride;
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
            const float floor = unorder(__reduce_min_sync(kAll, top[lane & (kBeamWarps - 1)]));
            for (int i = 0; i < n; i += 32) {
                const float cx = i + lane < n ? cand_x[warp][i + lane] : -CUDART_INF_F;
                best.offer(cx, i + lane < n && cx >= floor ? cand_v[warp][i + lane] : -1, K, lane);
            }
            __syncwarp();
            if (lane == 0)
                n_cand[warp] = 0;
            if (K > kBeamWarps && lane == (K - 1) / kBeamWarps)
                top[warp] = order(best.x);
            __syncwarp();
        };
        float R = -CUDART_INF_F, s = 0.f;
        int c = (split * kBeamWarps + warp) * kStep;
        const int stride = p.splits * kBeamWarps * kStep;
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
            float cm = -CUDART_INF_F;       // (fmaxf drops NaN)
#pragma unroll
            for (int j = 0; j < kLaneTok; ++j)
                cm = fmaxf(cm, x[j]);
            // sum of 2^(x log2 e - 4 R), R the lane's own running reference
            const float rn = fmaxf(R, cm * kLog2e4);
            if (fabsf(rn) < kLarge * kLog2e4) {
                const uint64_t c2 = pack2(kLog2e, kLog2e), r2 = pack2(-4.f * rn, -4.f * rn);
                uint64_t acc = 0;
#pragma unroll
                for (int j = 0; j < kLaneTok; j += 2) {
                    const float2 z = unpack2(fma2(pack2(x[j], x[j + 1]), c2, r2));
                    acc = add2(acc, pack2(ex2(z.x), ex2(z.y)));
                }
                const float2 a = unpack2(acc);
                s = (R > -CUDART_INF_F ? s * apart(R, rn) : s) + (a.x + a.y);
                R = rn;
            } else {
                // a largest logit from kLarge on, of either sign, or -inf alone, or NaN or +inf, which
                // have to show in the sum
                const float rm = cm > -CUDART_INF_F ? fmaxf(R, reference(cm)) : R;
                s = R > -CUDART_INF_F ? s * apart(R, rm) : s;
                R = rm;
#pragma unroll
                for (int j = 0; j < kLaneTok; ++j)
                    s += x[j] > -CUDART_INF_F ? apart(reference(x[j]), rm) : x[j] == x[j] ? 0.f : CUDART_NAN_F;
            }
            // Tokens that beat the K-th best so far. A warp's first chunk starts the list with
            // every lane's best; the others that may still beat it wait in shared memory until there
            // are 32 of them or the row ends (inserted chunk by chunk, each a chain of shuffles, they
            // took 9 of 35 us in 256 rows of 128001 tokens).
            // What all warps of the CTA hold is a bound, too: top[w] is the ceil(K / 8)-th best that
            // warp w has seen, so at least K tokens are as high as the lowest of them (read without
            // a barrier: an older value is only a weaker bound).
            const float floor = unorder(__reduce_min_sync(kAll, top[lane & (kBeamWarps - 1)]));
            if (__any_sync(kAll, cm >= floor && (cm > best.tx || best.tv < 0))) {
                const int v0 = (c + lane) * V - shift;
                // (tokens grow with j, so the first of equal logits is the lowest token)
                auto token = [&](int j) { return v0 + 32 * V * (j / V) + j % V; };
                if (K <= kBeamWarps) {
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
        insert_waiting();
        // the warp's reference and sum
        float wm = R;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            wm = fmaxf(wm, __shfl_xor_sync(kAll, wm, o));
        float ws = s == 0.f ? 0.f : wm > -CUDART_INF_F ? s * apart(R, wm) : s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            ws += __shfl_xor_sync(kAll, ws, o);
        if (lane == 0) {
            sh_m[warp] = wm;
            sh_s[warp] = ws;
        }
        // the CTA's best: all warps' j-th before any (j + 1)-th, so that the first 32 settle most
        if (lane < K) {
            sh_x[lane][warp] = best.x;
            sh_v[lane][warp] = best.v;
        }
        __syncthreads();
        if (warp == 0) {
            best.start((&sh_x[0][0])[lane], lane < K * kBeamWarps ? (&sh_v[0][0])[lane] : -1, K, lane);
            for (int i = 32; i < K * kBeamWarps; i += 32)
                best.offer((&sh_x[0][0])[i + lane], i + lane < K * kBeamWarps ? (&sh_v[0][0])[i + lane] : -1,
                           K, lane);
        }
        const size_t part = static_cast<size_t>(row) * p.splits + split;
        if (warp == 0) {
            float bm = lane < kBeamWarps ? sh_m[lane] : -CUDART_INF_F;
            const float mine = bm;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                bm = fmaxf(bm, __shfl_xor_sync(kAll, bm, o));
            float bs = lane < kBeamWarps ? sh_s[lane] : 0.f;
            bs = bs == 0.f ? 0.f : bm > -CUDART_INF_F ? bs * apart(mine, bm) : bs;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                bs += __shfl_xor_sync(kAll, bs, o);
            if (lane == 0)
                p.part_stat[part] = make_float2(bm, bs);
            if (lane < K) {
                const size_t at = (static_cast<size_t>(row) * K + lane) * p.splits + split;
                p.part_x[at] = best.x;
                p.part_v[at] = best.v;
            }
            __threadfence();
        }
    }
    // the last CTA of the group joins
    __syncthreads();
    if (tid == 0)
        sh_last = atomic_add_acq_rel_gpu(p.tickets + group, 1) == K * p.splits - 1;
    __syncthreads();
    if (!sh_last)
        return;
    __threadfence();
    if (tid == 0)
        p.tickets[group] = 0;
    // a warp per row: its statistics, its best tokens and their scores
    for (int b = warp; b < K; b += kBeamWarps) {
        const int r = group * K + b;
        const float cum = p.cum[r], scale = p.rank_scale ? p.rank_scale[r] : 1.f;
        const bool fin = p.done && p.done[r];
        // (requested together; a finished row's are not there and not used)
        const size_t part = static_cast<size_t>(r) * p.splits, list = part * K;
        const int n = p.splits * K;
        const float cx = lane < n ? __ldcg(p.part_x + list + lane) : 0.f;
        const int cv = lane < n ? __ldcg(p.part_v + list + lane) : -1;
        Best best;
        best.clear();
        float score = -CUDART_INF_F;
        if (fin) {
            if (lane == 0) {
                best.v = p.eos;
                score = isfinite(cum) ? cum : -CUDART_INF_F;
            }
        } else {
            float m = -CUDART_INF_F, s = 0.f;
            for (int i = lane; i < p.splits; i += 32) {
                const float2 st = __ldcg(p.part_stat + part + i);
                const float mn = fmaxf(m, st.x);
                if (st.y != 0.f) {
                    const float add = mn > -CUDART_INF_F ? st.y * apart(st.x, mn) : st.y;
                    s = (s != 0.f && mn > -CUDART_INF_F ? s * apart(m, mn) : s) + add;
                    m = mn;
                }
            }
            float wm = m;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                wm = fmaxf(wm, __shfl_xor_sync(kAll, wm, o));
            s = s == 0.f ? 0.f : wm > -CUDART_INF_F ? s * apart(m, wm) : s;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                s += __shfl_xor_sync(kAll, s, o);
            const float ls = logf(s);
            const bool dead = !isfinite(wm) || !isfinite(ls) || !isfinite(cum);
            if (dead) {
                best.v = lane < K && lane < p.vocab ? lane : -1;
            } else {
                // all splits' j-th before any (j + 1)-th
                for (int i = 0; i < n; i += 32) {
                    const float ox = i == 0 ? cx : i + lane < n ? __ldcg(p.part_x + list + i + lane) : 0.f;
                    const int ov = i == 0 ? cv : i + lane < n ? __ldcg(p.part_v + list + i + lane) : -1;
                    if (i == 0)
                        best.start(ox, ov, K, lane);
                    else
                        best.offer(ox, ov, K, lane);
                }
                // x - 4 R / kLog2e in double: in fp32 it would round at the size of the logits. From
                // kLarge on the largest logit, the list's first, stands for its reference.
                const float first = __shfl_sync(kAll, best.x, 0);
                if (best.v >= 0) {
                    const double ref = fabsf(wm) < kLarge * kLog2e4 ? wm / static_cast<double>(kLog2e4) : first;
                    score = static_cast<float>(best.x - ref - ls + cum);
                }
            }
        }
        if (lane < K) {
            row_s[b][lane] = score;
            row_x[b][lane] = score * scale;
            row_v[b][lane] = best.v;
        }
        if (lane == 0)
            row_done[b] = fin ? 1 : 0;
    }
    __syncthreads();
    // the group's best: candidate id = row * 16 + place in the row, so that ties by score go to
    // the lower row, and within a row to the higher logit, then the lower token
    if (warp == 0) {
        Best best;
        best.clear();
        // (place by place over the rows: the first 32 settle most)
        for (int i = 0; i < K * K; i += 32) {
            const int at = i + lane, j = at / K, b = at - j * K;
            const bool on = at < K * K && row_v[min(b, kMaxBeams - 1)][min(j, kMaxBeams - 1)] >= 0;
            const float ox = on ? row_x[b][j] : 0.f;
            if (i == 0)
                best.start(ox, on ? b * kMaxBeams + j : -1, K, lane);
            else
                best.offer(ox, on ? b * kMaxBeams + j : -1, K, lane);
        }
        if (lane < K) {
            const int id = max(best.v, 0);   // (all places are filled unless a scale is not a number)
            const int b = id / kMaxBeams, j = id % kMaxBeams, o = group * K + lane;
            const int token = row_v[b][j];
            p.parent[o] = group * K + b;
            p.token[o] = token;
            p.cum_out[o] = row_s[b][j];
            if (p.done_out)
                p.done_out[o] = row_done[b] || token == p.eos ? 1 : 0;
        }
    }
}

}  // namespace

cudaError_t launch_beam_select(const BeamParams &p, cudaStream_t stream)
{
    const dim3 grid(p.splits, p.n_groups * p.n_beams), block(kBeamThreads);
    const cudaError_t e = p.logits_fp32 ? launch_pdl(beam_kernel<float>, grid, block, 0, stream, p)
                                        : launch_pdl(beam_kernel<__nv_bfloat16>, grid, block, 0, stream, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sfi
