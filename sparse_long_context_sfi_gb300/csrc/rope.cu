// rope.cu -- rotary positions of the rows on their way to the cache, with the per-head norm in front
// of them: pairs (a, b) of a head's dimensions turned by the row's position,
//     y_a = c (x_a cos - x_b sin),  y_b = c (x_b cos + x_a sin),
// and the turned keys, and the values, put into their cache rows.
//
// The angle of pair i at position P is P * f_i turns. In 64-bit fixed point (units of 2^-64 turn) the
// product is exact modulo one turn, so far positions cost no range reduction and lose nothing:
// its upper half is the angle, in half turns as a float for sincospif.
//
// Bytes bound it: a row of a head is read and written once. A half-warp holds a row of a head, 8
// dimensions (16 bytes) a lane. A CTA has the sines and cosines of its rows in shared memory, worked
// out once for all heads and layers, and each half-warp keeps its row's in registers over the heads
// it goes through.
#include "chunk.cuh"
#include "sfi_device.cuh"

namespace sfi {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = kRopeThreads / 16;    // most rows of a CTA
constexpr int kRopeLoads = 4;                   // heads of a half-warp on their way at once
constexpr uint32_t kEvery = 0xffffffffu;

// How a lane gets the partners of its 8 dimensions.
enum {
    kPairs,     // neighbours: its own
    kLanes,     // half a head apart, a multiple of 8: all in one other lane
    kAnywhere   // any other distance: read again, one by one
};

__device__ __forceinline__ void unpack8(const uint4 &w, float *x)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A lane's share of the rotation: y = x * c + (partner) * s, weights of the norm included.
struct Turn {
    float c[8], s[8];
};

template <int MODE, bool NORM>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, int lg_rows, int need)
{
    __shared__ float2 cs[kRopeRows][kHeadDim / 2];
    __shared__ long long place[kRopeRows];
    __shared__ int at[kRopeRows];
    __shared__ bool live[kRopeRows];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_here = 1 << lg_rows, r0 = blockIdx.x << lg_rows;
    const int hq = p.q ? p.n_q_heads : 0, hkv = p.c.pg.n_kv_heads, hk = p.k ? hkv : 0;
    const bool append = p.k_cache != nullptr;
    const int half = p.rot >> 1;
    pdl_trigger();
    pdl_wait();
    // (what an append skips is told when the lengths advance)
    if (!append && blockIdx.x == 0 && blockIdx.y == 0) {
        for (int b = warp; b < p.c.pg.batch; b += kRopeThreads / 32) {
            int s0, n, L;
            if (p.c.pg.active && !p.c.pg.active[b])
                continue;
            if (need == kNeedLength)
                chunk_ok<kNeedLength>(p.c, b, lane, s0, n, L, lane == 0);
            else
                chunk_ok<kNeedRows>(p.c, b, lane, s0, n, L, lane == 0);
        }
    }
    for (int i = warp; i < n_here; i += kRopeThreads / 32) {
        const int r = r0 + i;
        int pos = 0;
        const int b = need == kNeedRoom     ? chunk_seq<kNeedRoom>(p.c, r, lane, pos)
                      : need == kNeedLength ? chunk_seq<kNeedLength>(p.c, r, lane, pos)
                                            : chunk_seq<kNeedRows>(p.c, r, lane, pos);
        if (lane == 0) {
            live[i] = b >= 0;
            at[i] = b < 0 ? 0 : p.pos ? p.pos[r] : pos;
            place[i] = append && b >= 0 ? cache_row(p.c.pg, b, pos) : -1;
        }
    }
    __syncthreads();
    for (int i = tid; i < half << lg_rows; i += kRopeThreads) {
        const int row = i / half, pair = i - row * half;
        const uint64_t turn = static_cast<uint64_t>(static_cast<long long>(at[row])) * p.turns[pair];
        float sn, cn;
        sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sn, &cn);
        cs[row][pair] = make_float2(cn * p.amplitude, sn * p.amplitude);
    }
    __syncthreads();

    const int hw = tid >> 4, l = tid & 15, row = hw & (n_here - 1), r = r0 + row;
    const bool on = live[row];
    // the partner's dimension and the factors of each of this lane's 8
    uint32_t turns8 = 0;            // which of them turn
    auto partner = [&](int d) {
        return MODE == kPairs ? d ^ 1 : d < half ? d + half : d - half;
    };
    auto factors = [&](const void *weight) {
        Turn t;
        const __nv_bfloat16 *w = static_cast<const __nv_bfloat16 *>(weight);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int d = 8 * l + j;
            const bool turned = d < p.rot;
            const int pair = MODE == kPairs ? d >> 1 : d < half ? d : d - half;
            const bool first = MODE == kPairs ? (d & 1) == 0 : d < half;
            const float2 v = turned ? cs[row][pair] : make_float2(1.f, 0.f);
            const float self = NORM && w ? __bfloat162float(w[d]) : 1.f;
            const float other = NORM && w && turned ? __bfloat162float(w[partner(d)]) : 1.f;
            t.c[j] = v.x * self;
            t.s[j] = (first ? -v.y : v.y) * other;
            turns8 |= turned ? 1u << j : 0u;
        }
        return t;
    };
    const Turn tq = factors(p.q_norm);
    const Turn tk = NORM ? factors(p.k_norm) : tq;
    const int other_lane = MODE == kLanes && 8 * l < p.rot ? (8 * l < half ? l + half / 8 : l - half / 8) : l;

    const int heads = hq + hk + (append ? hkv : 0), units = heads * p.n_layers;
    const int subs = kRopeRows >> lg_rows, stride = subs * gridDim.y;
    const int first = (hw >> lg_rows) * gridDim.y + blockIdx.y;
    const long long head = append ? (p.c.pg.page_size ? 16 : p.c.pg.capacity) : 1;
    const long long layer_rows = append ? (p.c.pg.page_size ? 16LL * p.c.pg.n_pages : 1LL * p.c.pg.batch * p.c.pg.capacity) * hkv : 0;
    // (both half-warps of a warp go through the same number of steps: shuffles)
    for (int u0 = 0; u0 < units; u0 += stride * kRopeLoads) {
        uint4 x[kRopeLoads];
        const __nv_bfloat16 *src[kRopeLoads];
        __nv_bfloat16 *dst[kRopeLoads];
        int kind[kRopeLoads];       // 0 q, 1 k, 2 v
#pragma unroll
        for (int i = 0; i < kRopeLoads; ++i) {
            const int u = u0 + first + i * stride;
            src[i] = nullptr;
            dst[i] = nullptr;
            kind[i] = 2;
            x[i] = make_uint4(0, 0, 0, 0);
            if (!on || u >= units)
                continue;
            const int layer = p.n_layers == 1 ? 0 : u / heads, h = u - layer * heads;
            const long long packed = static_cast<long long>(layer) * p.c.n_rows + r;
            if (h < hq) {
                kind[i] = 0;
                src[i] = static_cast<const __nv_bfloat16 *>(p.q) + packed * p.q_stride + h * kHeadDim;
                dst[i] = static_cast<__nv_bfloat16 *>(p.q_out) + (packed * hq + h) * kHeadDim;
            } else {
                const bool is_k = h < hq + hk;
                const int g = h - hq - (is_k ? 0 : hk);
                kind[i] = is_k ? 1 : 2;
                src[i] = is_k ? static_cast<const __nv_bfloat16 *>(p.k) + packed * p.k_stride + g * kHeadDim
                              : static_cast<const __nv_bfloat16 *>(p.v) + packed * p.v_stride + g * kHeadDim;
                if (!append)
                    dst[i] = static_cast<__nv_bfloat16 *>(p.k_out) + (packed * hkv + g) * kHeadDim;
                else if (place[row] >= 0)
                    dst[i] = static_cast<__nv_bfloat16 *>(is_k ? p.k_cache : p.v_cache) +
                             (layer * layer_rows + place[row] + g * head) * kHeadDim;
            }
            x[i] = __ldcs(reinterpret_cast<const uint4 *>(src[i]) + l);
        }
#pragma unroll
        for (int i = 0; i < kRopeLoads; ++i) {
            float a[8], b[8];
            unpack8(x[i], a);
            if constexpr (MODE == kLanes) {
                const uint4 o = make_uint4(__shfl_sync(kEvery, x[i].x, other_lane, 16),
                                           __shfl_sync(kEvery, x[i].y, other_lane, 16),
                                           __shfl_sync(kEvery, x[i].z, other_lane, 16),
                                           __shfl_sync(kEvery, x[i].w, other_lane, 16));
                unpack8(o, b);
            } else if constexpr (MODE == kAnywhere) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int d = 8 * l + j;
                    b[j] = src[i] && d < p.rot ? __bfloat162float(src[i][partner(d)]) : 0.f;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    b[j] = a[j ^ 1];
            }
            float scale = 1.f;
            if constexpr (NORM) {
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    sum = fmaf(a[j], a[j], sum);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1)
                    sum += __shfl_xor_sync(kEvery, sum, o, 16);
                if (kind[i] == 0 ? p.q_norm != nullptr : p.k_norm != nullptr)
                    scale = rsqrtf(sum * (1.f / kHeadDim) + p.eps);
            }
            if (kind[i] < 2) {
                const Turn &t = NORM && kind[i] == 1 ? tk : tq;
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    // (a dimension that stays has no partner whose infinity could reach it)
                    const float own = a[j] * t.c[j];
                    y[j] = (turns8 >> j) & 1u ? fmaf(b[j], t.s[j], own) : own;
                    if (NORM)
                        y[j] *= scale;
                }
                x[i] = make_uint4(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]), bf16_pair(y[4], y[5]),
                                  bf16_pair(y[6], y[7]));
            }
        }
        __syncwarp();               // in place, partners have been read
#pragma unroll
        for (int i = 0; i < kRopeLoads; ++i)
            if (dst[i])
                reinterpret_cast<uint4 *>(dst[i])[l] = x[i];
    }
}

template <int MODE>
cudaError_t launch_mode(const RopeParams &p, dim3 grid, int lg_rows, int need, cudaStream_t stream)
{
    return p.q_norm || p.k_norm
               ? launch_pdl(rope_kernel<MODE, true>, grid, dim3(kRopeThreads), 0, stream, p, lg_rows, need)
               : launch_pdl(rope_kernel<MODE, false>, grid, dim3(kRopeThreads), 0, stream, p, lg_rows, need);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, int sms, cudaStream_t stream)
{
    const bool append = p.k_cache != nullptr;
    const int hkv = p.c.pg.n_kv_heads;
    const int units = ((p.q ? p.n_q_heads : 0) + (p.k ? hkv : 0) + (append ? hkv : 0)) * p.n_layers;
    // The most rows per CTA that still fill the GPU, and then CTAs that share a row's heads.
    int lg = 4;
    while (lg > 0 && (p.c.n_rows >> lg) < 2 * sms)
        --lg;
    const int blocks = (p.c.n_rows + (1 << lg) - 1) >> lg, subs = kRopeRows >> lg;
    int share = 4 * sms / blocks;
    const int most = (units + subs - 1) / subs;
    share = share < most ? share : most;
    const dim3 grid(blocks, share < 1 ? 1 : share);
    const int need = append ? kNeedRoom : p.pos ? kNeedRows : kNeedLength;
    const int half = p.rot / 2;
    cudaError_t e = p.interleaved   ? launch_mode<kPairs>(p, grid, lg, need, stream)
                    : half % 8 == 0 ? launch_mode<kLanes>(p, grid, lg, need, stream)
                                    : launch_mode<kAnywhere>(p, grid, lg, need, stream);
    if (e == cudaSuccess && append)
        return launch_advance(p.c, stream);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sfi
