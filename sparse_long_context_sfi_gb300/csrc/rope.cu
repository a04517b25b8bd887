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
// dimensions (16 bytes) a lane, 4 heads on their way at once. A CTA has the sines and cosines of its 8
// rows in shared memory, worked out once for all heads, and each half-warp keeps its row's share in
// registers over the heads it goes through, multiplied by the norm's weights.
// Four prompts of 8192 tokens, 32 and 8 heads: 131 us, 6.15 TB/s (copy rate 6.75), with norms 138, with
// neighbouring pairs 129, with 40 of 128 dimensions 135 (209 with the partners read again from the
// cache), with 66 145; 170 us with 16 rows a CTA, unpacked arithmetic and a list of (layer, head) per
// step; 135 for 133 with 80 instead of 64 registers; 178 (148 with 80 registers) where a head's place
// is loaded again as soon as the head is stored.
#include "chunk.cuh"
#include "sfi_device.cuh"

namespace sfi {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 8;                    // most rows of a CTA: one for each warp to look up
constexpr int kRopeLoads = 4;                   // heads of a half-warp on their way at once
constexpr uint32_t kEvery = 0xffffffffu;

// How a lane gets the partners of its 8 dimensions.
enum {
    kPairs,     // neighbours: its own
    kLanes,     // half of rot_dim apart, a multiple of 8: all in one other lane
    kAnywhere   // half of any other rot_dim apart: through shared memory
};

__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ float2 unpack2(uint64_t v)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Two bf16 as two floats.
__device__ __forceinline__ uint64_t widen(uint32_t u)
{
    return pack2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

__device__ __forceinline__ uint32_t narrow(uint64_t v)
{
    const float2 f = unpack2(v);
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A lane's share of the rotation: y = x * c + (partner) * s, weights of the norm included.
struct Turn {
    uint64_t c[4], s[4];
};

template <int MODE, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const RopeParams p, int lg_rows, int need, int fused)
{
    __shared__ __align__(16) float2 cs[kRopeRows][kHeadDim / 2];
    __shared__ long long place[kRopeRows];
    __shared__ int at[kRopeRows];
    __shared__ bool live[kRopeRows];
    __shared__ uint4 held[MODE == kAnywhere ? kRopeThreads * kRopeLoads : 1];   // the heads on their way
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_here = 1 << lg_rows, r0 = blockIdx.x << lg_rows, layer = blockIdx.z;
    const int hkv = p.c.pg.n_kv_heads, hq = p.q ? p.n_q_heads : 0, hk = p.k ? hkv : 0;
    const bool append = p.k_cache != nullptr;
    const int half = p.rot >> 1;
    // half-warps: row hw % n_here, and of its heads every `stride`-th from `u` on
    const int hw = tid >> 4, l = tid & 15, row = hw & (n_here - 1), r = r0 + row;
    const int stride = ((kRopeThreads / 16) >> lg_rows) * gridDim.y;
    int u = (hw >> lg_rows) * gridDim.y + blockIdx.y;
    const long long packed = static_cast<long long>(layer) * p.c.n_rows + r;
    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(p.q) + packed * p.q_stride + 8 * l;
    const bool there = r < p.c.n_rows;
    pdl_trigger();
    pdl_wait();
    // the first queries are asked for before their positions are known (a chain of four loads)
    uint4 x[kRopeLoads];
    auto load = [&](const __nv_bfloat16 *from, int begin, int end, bool on) {
#pragma unroll
        for (int i = 0; i < kRopeLoads; ++i) {
            const int h = u + i * stride - begin;
            x[i] = on && h < end - begin ? __ldcs(reinterpret_cast<const uint4 *>(from + h * kHeadDim))
                                         : make_uint4(0, 0, 0, 0);
        }
    };
    load(src, 0, hq, there);
    // (what an append skips is told when the lengths advance)
    if (!append && blockIdx.x == 0 && blockIdx.y == 0 && layer == 0) {
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
    if (warp < n_here) {
        const int mine = r0 + warp;
        int pos = 0;
        const int b = need == kNeedRoom     ? chunk_seq<kNeedRoom>(p.c, mine, lane, pos)
                      : need == kNeedLength ? chunk_seq<kNeedLength>(p.c, mine, lane, pos)
                                            : chunk_seq<kNeedRows>(p.c, mine, lane, pos);
        if (lane == 0) {
            live[warp] = b >= 0;
            at[warp] = b < 0 ? 0 : p.pos ? p.pos[mine] : pos;
            place[warp] = append && b >= 0 ? cache_row(p.c.pg, b, pos) : -1;
        }
    }
    __syncthreads();
    for (int i = tid; i < half << lg_rows; i += kRopeThreads) {
        const int which = i / half, pair = i - which * half;
        const uint64_t turn = static_cast<uint64_t>(static_cast<long long>(at[which])) * p.turns[pair];
        float sn, cn;
        sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sn, &cn);
        cs[which][pair] = make_float2(cn * p.amplitude, sn * p.amplitude);
    }
    __syncthreads();

    const bool on = live[row];
    const bool turns = 8 * l < p.rot;       // some of its dimensions (kLanes: all)
    constexpr bool pairs = MODE == kPairs;
    auto partner = [&](int d) { return pairs ? d ^ 1 : d < half ? d + half : d - half; };
    const int other_lane = MODE == kLanes && turns ? (8 * l < half ? l + half / 8 : l - half / 8) : l;
    auto factors = [&](const void *weight) {
        Turn t;
        float c[8], s[8];
        if constexpr (MODE == kAnywhere) {
            const __nv_bfloat16 *w = static_cast<const __nv_bfloat16 *>(weight);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int d = 8 * l + j;
                const bool turned = d < p.rot;
                // (a dimension that stays adds 0 * -0 = -0, which leaves a -0 as it is, too)
                const float2 v = turned ? cs[row][d < half ? d : d - half] : make_float2(1.f, -0.f);
                c[j] = NORM && w ? v.x * __bfloat162float(w[d]) : v.x;
                s[j] = (d < half ? -v.y : v.y) * (NORM && w && turned ? __bfloat162float(w[partner(d)]) : 1.f);
            }
        } else {
            // (16 bytes at a time; the lane's first pair is a multiple of 4, or of 8)
            const uint4 *w = static_cast<const uint4 *>(weight);
            const int pair = pairs ? 4 * l : 8 * l < half ? 8 * l : 8 * l - half;
            const float4 *v = reinterpret_cast<const float4 *>(cs[row] + (turns ? pair : 0));
            uint4 own = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u), other = own;
            if (NORM && w) {
                own = w[l];
                other = pairs ? own : w[other_lane];
            }
            const uint32_t wo[4] = {own.x, own.y, own.z, own.w}, wt[4] = {other.x, other.y, other.z, other.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float4 f;               // cosine, sine of the two dimensions
                if (pairs) {
                    const float4 g = v[j / 2];
                    f = j % 2 == 0 ? make_float4(g.x, -g.y, g.x, g.y) : make_float4(g.z, -g.w, g.z, g.w);
                } else {
                    const float4 g = v[j];
                    f = 8 * l < half ? make_float4(g.x, -g.y, g.z, -g.w) : g;
                }
                if (!(pairs ? 8 * l + 2 * j < p.rot : turns))
                    f = make_float4(1.f, 0.f, 1.f, 0.f);
                const float2 a = unpack2(widen(wo[j])), b = unpack2(widen(wt[j]));
                c[2 * j] = f.x * a.x;
                c[2 * j + 1] = f.z * a.y;
                s[2 * j] = f.y * (pairs ? b.y : b.x);
                s[2 * j + 1] = f.w * (pairs ? b.x : b.y);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            t.c[j] = pack2(c[2 * j], c[2 * j + 1]);
            t.s[j] = pack2(s[2 * j], s[2 * j + 1]);
        }
        return t;
    };
    // The heads [begin, end) of the row, which lie at `from` and go to `to`, to_step elements apart; TURN:
    // turned by t (and normed), else copied. Both half-warps of a warp go through as many steps.
    auto heads = [&](int begin, int end, const __nv_bfloat16 *from, __nv_bfloat16 *to, long long to_step, bool turn,
                     const Turn &t, bool norm, bool loaded) {
        while (__any_sync(kEvery, u < end)) {
            if (!loaded)
                load(from, begin, end, on);
            loaded = false;
            if (turn) {
                if constexpr (MODE == kAnywhere) {
                    __syncwarp();               // the last heads have been read
#pragma unroll
                    for (int i = 0; i < kRopeLoads; ++i)
                        held[(hw * kRopeLoads + i) * 16 + l] = x[i];
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < kRopeLoads; ++i) {
                    if (MODE != kAnywhere && !__any_sync(kEvery, u + i * stride < end))
                        break;
                    const uint64_t a[4] = {widen(x[i].x), widen(x[i].y), widen(x[i].z), widen(x[i].w)};
                    uint64_t b[4], y[4];
                    if constexpr (MODE == kLanes) {
                        b[0] = widen(__shfl_sync(kEvery, x[i].x, other_lane, 16));
                        b[1] = widen(__shfl_sync(kEvery, x[i].y, other_lane, 16));
                        b[2] = widen(__shfl_sync(kEvery, x[i].z, other_lane, 16));
                        b[3] = widen(__shfl_sync(kEvery, x[i].w, other_lane, 16));
                    } else if constexpr (MODE == kPairs) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 f = unpack2(a[j]);
                            b[j] = pack2(f.y, f.x);
                        }
                    } else {
                        // (0 where a dimension stays: no infinity reaches it)
                        const __nv_bfloat16 *from_row = reinterpret_cast<const __nv_bfloat16 *>(held + (hw * kRopeLoads + i) * 16);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int d = 8 * l + 2 * j;
                            if (half % 2 == 0) {        // both on the same side, and aligned
                                b[j] = d < p.rot ? widen(*reinterpret_cast<const uint32_t *>(from_row + partner(d))) : 0;
                            } else {
                                b[j] = d < p.rot ? pack2(__bfloat162float(from_row[partner(d)]),
                                                         __bfloat162float(from_row[partner(d + 1)])) : 0;
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        y[j] = mul2(a[j], t.c[j]);
                        // (rot_dim is even: neighbours turn, or stay, together)
                        if (MODE == kAnywhere || (MODE == kLanes ? turns : 8 * l + 2 * j < p.rot))
                            y[j] = fma2(b[j], t.s[j], y[j]);
                    }
                    if constexpr (NORM) {
                        uint64_t sq = mul2(a[0], a[0]);
#pragma unroll
                        for (int j = 1; j < 4; ++j)
                            sq = fma2(a[j], a[j], sq);
                        const float2 f = unpack2(sq);
                        float sum = f.x + f.y;
#pragma unroll
                        for (int o = 8; o > 0; o >>= 1)
                            sum += __shfl_xor_sync(kEvery, sum, o, 16);
                        const float scale = norm ? rsqrtf(sum * (1.f / kHeadDim) + p.eps) : 1.f;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            y[j] = mul2(y[j], pack2(scale, scale));
                    }
                    x[i] = make_uint4(narrow(y[0]), narrow(y[1]), narrow(y[2]), narrow(y[3]));
                }
            }
#pragma unroll
            for (int i = 0; i < kRopeLoads; ++i) {
                const int h = u + i * stride - begin;
                if (on && to && h < end - begin)
                    *reinterpret_cast<uint4 *>(to + h * to_step) = x[i];
            }
            // (kRopeLoads * stride may pass the end: the next heads begin where this class goes on)
#pragma unroll
            for (int i = 0; i < kRopeLoads; ++i)
                u += u < end ? stride : 0;
        }
    };
    Turn t = factors(p.q_norm);
    if (hq > 0)
        heads(0, hq, src, static_cast<__nv_bfloat16 *>(p.q_out) + packed * hq * kHeadDim + 8 * l, kHeadDim, true, t,
              p.q_norm != nullptr, true);
    if (hk > 0) {
        if (NORM)
            t = factors(p.k_norm);
        long long step = kHeadDim;
        __nv_bfloat16 *k_to, *v_to = nullptr;
        if (append) {
            step = (p.c.pg.page_size ? 16LL : p.c.pg.capacity) * kHeadDim;
            const long long rows = p.c.pg.page_size ? 16LL * p.c.pg.n_pages : 1LL * p.c.pg.batch * p.c.pg.capacity;
            const long long to = (layer * rows * hkv + place[row]) * kHeadDim + 8 * l;
            k_to = place[row] < 0 ? nullptr : static_cast<__nv_bfloat16 *>(p.k_cache) + to;
            v_to = place[row] < 0 ? nullptr : static_cast<__nv_bfloat16 *>(p.v_cache) + to;
        } else {
            k_to = static_cast<__nv_bfloat16 *>(p.k_out) + packed * hkv * kHeadDim + 8 * l;
        }
        heads(hq, hq + hk, static_cast<const __nv_bfloat16 *>(p.k) + packed * p.k_stride + 8 * l, k_to, step, true, t,
              p.k_norm != nullptr, false);
        if (append)
            heads(hq + hk, hq + 2 * hk, static_cast<const __nv_bfloat16 *>(p.v) + packed * p.v_stride + 8 * l, v_to,
                  step, false, t, false, false);
    }
    if (fused > 0) {            // all of the grid, one cluster, has read the lengths
        if (fused > 1)
            cluster_sync_all();
        if (fused == 1 || cluster_ctarank() == 0)
            advance_lengths(p.c);
    }
}

template <int MODE>
cudaError_t launch_mode(const RopeParams &p, dim3 grid, int lg_rows, int need, int fused, cudaStream_t stream)
{
    auto *kern = p.q_norm || p.k_norm ? rope_kernel<MODE, true> : rope_kernel<MODE, false>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;       // (the whole grid)
    attr[1].val.clusterDim.x = grid.x;
    attr[1].val.clusterDim.y = grid.y;
    attr[1].val.clusterDim.z = grid.z;
    cfg.attrs = attr;
    cfg.numAttrs = fused > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p, lg_rows, need, fused);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, int sms, cudaStream_t stream)
{
    const bool append = p.k_cache != nullptr;
    const int hkv = p.c.pg.n_kv_heads;
    const int heads = (p.q ? p.n_q_heads : 0) + (p.k ? hkv : 0) + (append ? hkv : 0);
    // The most rows per CTA that still fill the GPU, and then CTAs that share a row's heads.
    int lg = 3;
    while (lg > 0 && (static_cast<long long>(p.c.n_rows) * p.n_layers >> lg) < 2 * sms)
        --lg;
    auto shape = [&](long long ctas) {
        const long long blocks = (p.c.n_rows + (1LL << lg) - 1) >> lg, subs = (kRopeThreads / 16) >> lg;
        const long long share = ctas / (blocks * p.n_layers), most = (heads + subs - 1) / subs;
        return dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(share < 1 ? 1 : share < most ? share : most),
                    p.n_layers);
    };
    dim3 grid = shape(4LL * sms);
    // A few tokens are one cluster, whose first CTA advances the lengths when all have read them: at
    // most 16 heads a half-warp, and a sequence for each of that CTA's warps. (One token of 12 heads: 6.2
    // us with the copy that resets the case, 8.2 in two launches; 4 of 48 8.2 and 8.9; 16, with two sequences
    // a warp, 10.2 and 9.6. The host issues one launch less.)
    int fused = 0;
    for (int i = 0; append && p.c.pg.batch <= 8 && fused == 0 && i <= 3; ++i) {
        const int keep = lg;
        lg = i;
        const dim3 g = shape(8);
        const unsigned n = g.x * g.y * g.z;
        if (n <= 8 && heads <= 16LL * ((kRopeThreads / 16) >> i) * g.y) {
            grid = g;
            fused = static_cast<int>(n);
        } else {
            lg = keep;
        }
    }
    const int need = append ? kNeedRoom : p.pos ? kNeedRows : kNeedLength;
    const cudaError_t e = p.interleaved       ? launch_mode<kPairs>(p, grid, lg, need, fused, stream)
                          : p.rot % 16 == 0 ? launch_mode<kLanes>(p, grid, lg, need, fused, stream)
                                            : launch_mode<kAnywhere>(p, grid, lg, need, fused, stream);
    if (e == cudaSuccess && append && fused == 0)
        return launch_advance(p.c, stream);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sfi
