// score.cu -- log probabilities of given tokens, with rank, entropy and the best alternatives, in one
// pass over the logits. With x = logits of a row and R a reference,
//     s = sum 2^(x log2 e - R),  t = sum (x log2 e - R) 2^(x log2 e - R),
//     lse = (R + log2 s) ln 2,   entropy = ln s - ln 2 * t / s,
// both kept relative to each lane's own running reference and moved by 2^(R - R') when that grows
// (t also by s (R - R')). The rank counts the tokens in front of the given one on the way.
//
// The bytes of the logits bound it, and right behind them issue slots: at the copy rate there are 11
// for a token of bf16. A pass over one takes 5.4 (unpacked, a packed multiply-add, an exponential, packed
// sums, half an instruction of a packed maximum, and its share of a chunk's loads and reference), the
// rank 1 (pairs compared, two comparisons added at once as integers), entropy 1.5, the list of the best
// a third: it is made behind the pass, of the few lanes whose highest chunks say that they hold one of
// them. What is left is a row's end, a chain of barriers, reductions and loads that come from HBM again:
// 8192 rows of 32000 bf16 take 84 us (6.2 TB/s) with the log probability alone, 90 with rank and entropy,
// 99 with 3 alternatives too, 117 with 20 (260 with a sorted list kept on the way, a comparison of two
// conditions per token for the rank and 8 warps per row); 2048 rows of 128001 85 us (6.2 TB/s); 256 rows of
// 128001 fp32 29 (4.5 TB/s) with rank and entropy, 36 with 20 alternatives. Tried: CTAs that go on to
// further rows, with the next row's first loads under way while one is finished (198 instead of 151
// then: spills, and warps that wait for the one that finishes; of one warp 111 for 99); mma.sync with ones to add up the rank's
// comparisons (124 for 120) and with the unit matrix to unpack bf16 (134).
#include "vocab.cuh"

#include <cfloat>
#include <climits>

namespace sfi {
namespace {

constexpr int kScoreWarps = 8;              // most warps of a CTA
// -150 is below every power that 32 bits hold: a term of it adds nothing, and 0 * -inf does not arise
constexpr float kNothing = -150.f;

// Sums of a set of tokens relative to their reference (in units of 2^4, see vocab.cuh).
struct Sums {
    float R, s, t;
    int front;
};

// The sums relative to a reference that is not below theirs; one that is not a number stays so.
template <bool ENT>
__device__ __forceinline__ Sums moved(const Sums &v, float R)
{
    Sums o = {R, 0.f, 0.f, v.front};
    if (v.s != 0.f) {
        const float d = R > -CUDART_INF_F ? 4.f * (v.R - R) : 0.f, w = ex2(d);
        o.s = v.s * w;
        if (ENT && w != 0.f)        // (d may be beyond what 32 bits hold)
            o.t = (v.t + v.s * d) * w;
    }
    return o;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// A lane's share of a chunk: four pieces of 16 bytes, 32 pieces apart, as they lie in memory. How its
// highest logit is found, how many tokens reach a threshold, and its terms of the sums.
template <typename T>
struct Part;

template <>
struct Part<float> {
    static constexpr int kV = 4;
    uint64_t n = 0;             // tokens counted, as floats (exact: a lane sees fewer than 2^24 of a row)

    static __device__ __forceinline__ float value(uint32_t u) { return __uint_as_float(u); }
    static __device__ __forceinline__ float highest(const uint4 *w)     // (max drops NaN)
    {
        float m = fmaxf(value(w[0].x), value(w[0].y));
        m = max3(m, value(w[0].z), value(w[0].w));
#pragma unroll
        for (int i = 1; i < 4; ++i)
            m = max3(max3(m, value(w[i].x), value(w[i].y)), value(w[i].z), value(w[i].w));
        return m;
    }
    __device__ __forceinline__ void count(const uint4 &w, float least)
    {
        float f[4];
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("set.ge.f32.f32 %0, %1, %2;" : "=f"(f[i]) : "f"(value(u[i])), "f"(least));
        n = add2(add2(n, pack2(f[0], f[1])), pack2(f[2], f[3]));
    }
    __device__ __forceinline__ void settle() {}
    __device__ __forceinline__ int counted() const
    {
        const float2 v = unpack2(n);
        return static_cast<int>(v.x) + static_cast<int>(v.y);
    }
    // the terms of one piece: powers into acc, and times their exponents into ent
    struct Low {
        __device__ __forceinline__ explicit Low(float) {}
    };
    template <bool ENT>
    static __device__ __forceinline__ void terms(const uint4 &w, Low, uint64_t c2, uint64_t r2, uint64_t &acc,
                                                 uint64_t &ent)
    {
        const uint64_t x[2] = {pack2(value(w.x), value(w.y)), pack2(value(w.z), value(w.w))};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 z = unpack2(fma2(x[i], c2, r2));
            const uint64_t e = pack2(ex2(z.x), ex2(z.y));
            acc = add2(acc, e);
            // (no 0 * -inf; a NaN is in acc)
            if (ENT)
                ent = fma2(e, pack2(fmaxf(z.x, kNothing), fmaxf(z.y, kNothing)), ent);
        }
    }
};

// Two tokens at a time where bf16 does: 16 instructions for 32 tokens' maximum, 32 to count them.
template <>
struct Part<__nv_bfloat16> {
    static constexpr int kV = 8;
    int n = 0;
    uint32_t chunk = 0;

    static __device__ __forceinline__ __nv_bfloat162 pair(uint32_t u) { return *reinterpret_cast<const __nv_bfloat162 *>(&u); }
    static __device__ __forceinline__ float highest(const uint4 *w)
    {
        __nv_bfloat162 m = __hmax2(__hmax2(pair(w[0].x), pair(w[0].y)), __hmax2(pair(w[0].z), pair(w[0].w)));
#pragma unroll
        for (int i = 1; i < 4; ++i)
            m = __hmax2(m, __hmax2(__hmax2(pair(w[i].x), pair(w[i].y)), __hmax2(pair(w[i].z), pair(w[i].w))));
        const float2 f = __bfloat1622float2(m);
        return fmaxf(f.x, f.y);
    }
    // (a pair's comparison is all ones in a half where it holds: less it, a sum has the lower halves that
    // hold in its lower half, and in its upper the upper less the lower ones)
    __device__ __forceinline__ void count(const uint4 &w, float least)
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        const __nv_bfloat162 l = __float2bfloat162_rn(least);       // (exact)
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c -= __hge2_mask(pair(u[i]), l);
        chunk += c;
    }
    __device__ __forceinline__ void settle()
    {
        n = __dp2a_lo(static_cast<int>(chunk), 0x0102, n);
        chunk = 0;
    }
    __device__ __forceinline__ int counted() const { return n; }
    // Logits below 150 powers under the reference are lifted to there (rounded down): they add
    // nothing either way, and -inf no 0 * -inf. NaN stays.
    struct Low {
        __nv_bfloat162 x;
        __device__ __forceinline__ explicit Low(float rn)
        {
            const __nv_bfloat16 l = __float2bfloat16_rd((4.f * rn + kNothing) * (1.f / kLog2e));
            x = __halves2bfloat162(l, l);
        }
    };
    template <bool ENT>
    static __device__ __forceinline__ void terms(const uint4 &w, const Low &low, uint64_t c2, uint64_t r2,
                                                 uint64_t &acc, uint64_t &ent)
    {
        uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (ENT) {
                const __nv_bfloat162 m = __hmax2_nan(pair(u[i]), low.x);
                u[i] = *reinterpret_cast<const uint32_t *>(&m);
            }
            const uint64_t z2 = fma2(pack2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u)), c2, r2);
            const float2 z = unpack2(z2);
            const uint64_t e = pack2(ex2(z.x), ex2(z.y));
            acc = add2(acc, e);
            if (ENT)
                ent = fma2(e, z2, ent);
        }
    }
};

// N 16-byte pieces of a row, 32 apart; pieces that reach over either end of the row are put together
// from its tokens, those beyond them are -inf, which no sum and no list sees.
template <typename T, int N>
__device__ __forceinline__ void load_pieces(const T *row, int shift, int vocab, int piece, uint4 *w)
{
    constexpr int V = Chunk<T>::kV;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = (piece + 32 * i) * V - shift;           // first token of the piece
        if (at >= 0 && at + V <= vocab) {
            w[i] = __ldcs(reinterpret_cast<const uint4 *>(row + at));
        } else if (at >= vocab || at + V <= 0) {
            const uint32_t low = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
            w[i] = make_uint4(low, low, low, low);
        } else {
            T t[V];
#pragma unroll
            for (int j = 0; j < V; ++j)
                t[j] = at + j >= 0 && at + j < vocab ? row[at + j] : static_cast<T>(-CUDART_INF_F);
            w[i] = *reinterpret_cast<const uint4 *>(t);
        }
    }
}

// A chunk that reaches over an end of the row.
template <typename T>
__device__ __noinline__ void load_edge(const T *row, int shift, int vocab, int piece, uint4 *w)
{
    load_pieces<T, 4>(row, shift, vocab, piece, w);
}

// The terms of a chunk whose reference is from kLarge on, of either sign, or whose highest logit is
// not a number that counts: what vocab.cuh says, one by one.
template <typename T>
__device__ __noinline__ Sums odd_chunk(Sums a, float cm, const uint4 *w)
{
    constexpr int V = Part<T>::kV;
    const float rm = cm > -CUDART_INF_F ? fmaxf(a.R, reference(cm)) : a.R;
    if (a.s != 0.f && rm > a.R) {
        const float d = 4.f * (a.R - rm), f = ex2(d);
        a.t = f != 0.f ? (a.t + a.s * d) * f : 0.f;
        a.s *= f;
    }
    a.R = rm;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        float x[V];
        Chunk<T>::unpack(w[i], x);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float z = 4.f * (reference(x[j]) - rm), e = ex2(z);
            a.s += x[j] > -CUDART_INF_F ? e : x[j] == x[j] ? 0.f : CUDART_NAN_F;
            if (e != 0.f && x[j] > -CUDART_INF_F)
                a.t += e * z;
        }
    }
    return a;
}

// The best K of a list b and n further candidates.
__device__ __noinline__ Best merged(Best b, const volatile float *x, const volatile int *v, int n, int K, int lane)
{
    for (int i = 0; i < n; i += 32) {
        const float cx = i + lane < n ? x[i + lane] : -CUDART_INF_F;
        const int cv = i + lane < n ? v[i + lane] : -1;
        // (a sort of the warp costs as much as about 12 insertions)
        if (i == 0 && n > 12 && b.tv < 0 && !__any_sync(kAll, b.v >= 0))
            b.start(cx, cv, K, lane);
        else
            b.offer(cx, cv, K, lane);
    }
    return b;
}

// The best K of up to 64 candidates: each one's place is the number of those before it (all
// comparisons at once, where insertions wait for one another). out_x and out_v hold K.
__device__ __noinline__ Best placed(const volatile float *x, const volatile int *v, int n, int K, int lane,
                                    volatile float *out_x, volatile int *out_v)
{
    const bool two = n > 32;
    const float x0 = lane < n ? x[lane] : -CUDART_INF_F, x1 = lane + 32 < n ? x[lane + 32] : -CUDART_INF_F;
    const int v0 = lane < n ? v[lane] : -1, v1 = lane + 32 < n ? v[lane + 32] : -1;
    int r0 = 0, r1 = 0;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const float ox = x[i];
        const int ov = v[i];
        r0 += better(ox, ov, x0, v0);
        if (two)
            r1 += better(ox, ov, x1, v1);
    }
    if (lane < n && r0 < K) {
        out_x[r0] = x0;
        out_v[r0] = v0;
    }
    if (lane + 32 < n && r1 < K) {
        out_x[r1] = x1;
        out_v[r1] = v1;
    }
    __syncwarp();
    Best b;
    b.x = lane < n && lane < K ? out_x[lane] : -CUDART_INF_F;
    b.v = lane < n && lane < K ? out_v[lane] : -1;
    b.tx = __shfl_sync(kAll, b.x, K - 1);
    b.tv = __shfl_sync(kAll, b.v, K - 1);
    return b;
}

// The lowest value of the type above x (not NaN).
__device__ __forceinline__ float above(float x, float)
{
    const int i = __float_as_int(x);
    return x == 0.f ? __int_as_float(1) : __int_as_float(i < 0 ? i - 1 : i + 1);
}
__device__ __forceinline__ float above(float x, __nv_bfloat16)
{
    const int i = __float_as_int(x);
    return x == 0.f ? __int_as_float(1 << 16) : __int_as_float(i < 0 ? i - (1 << 16) : i + (1 << 16));
}

// A row, or a split of one, as its CTA sees it.
template <typename T>
struct Place {
    const T *x;
    int shift, pieces;      // tokens in front of the row in its first 16-byte piece; pieces of the row
    int row, split;

    __device__ __forceinline__ Place(const ScoreParams &p, int item)
    {
        row = p.splits == 1 ? item : item / p.splits;
        split = item - row * p.splits;
        x = static_cast<const T *>(p.logits) + static_cast<size_t>(row) * p.row_stride;
        shift = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
        pieces = (p.vocab + shift + Chunk<T>::kV - 1) / Chunk<T>::kV;
    }
};

constexpr int kBuffer = 256;        // of the tokens that may be among the best

// A chunk's highest logit with the number of the chunk (of its warp's, from 0) in the low bits: all
// that bf16 leaves free, 12 of fp32's own. In order as the logits are, but for those that differ in
// these bits alone; what a key stands for lies between lo and hi. The last number says "this or a
// later one". (That of an infinity may be no number: -inf
// then; a row with +inf has no list.)
template <typename T>
struct Key {
    static constexpr uint32_t kNumber = sizeof(T) == 2 ? 0xffffu : 0xfffu;

    static __device__ __forceinline__ float of(float x, uint32_t number)
    {
        return __uint_as_float((__float_as_uint(x) & ~kNumber) | number);
    }
    static __device__ __forceinline__ uint32_t number(float k) { return __float_as_uint(k) & kNumber; }
    static __device__ __forceinline__ float least(float k) { return __uint_as_float(__float_as_uint(k) & ~kNumber); }
    static __device__ __forceinline__ float most(float k)
    {
        return sizeof(T) == 2 ? least(k) : __uint_as_float(__float_as_uint(k) | kNumber);
    }
    static __device__ __forceinline__ float lo(float k) { return signbit(k) ? most(k) : least(k); }
    static __device__ __forceinline__ float hi(float k) { return signbit(k) ? least(k) : most(k); }
};

// Every lane keeps its three highest chunks' keys. K lanes have a logit of `least`, the K-th highest
// lane's, or more, so all of the K best tokens do, and they lie in the lanes that reach it: few, of
// which the one or two chunks that do are read again, or where the third one does, too, all.
//
// At most 64, 72, 80 registers with rank and entropy, us: 8192 rows of 32000 bf16 with 3 tokens 109, 99,
// 111, without a list 95, 90, 100; of fp32 185, 178, 167 (80 allowed, 72 taken) and 169, 163, 181.
template <typename T, bool TOP, bool RANK, bool ENT>
__global__ void __maxnreg__(RANK && ENT ? (TOP && sizeof(T) == 4 ? 80 : 72) : 64) score_kernel(const ScoreParams p)
{
    // keys of every lane; lists of the best, the warps' own where the buffer is too small, in their place
    extern __shared__ __align__(16) float sh_top[];
    float *const lane_k = sh_top, *const sh_x = sh_top;
    int *const sh_v = reinterpret_cast<int *>(sh_x + blockDim.x);
    float *const cand_x = lane_k + 3 * blockDim.x;
    int *const cand_v = reinterpret_cast<int *>(cand_x + kBuffer);
    // lanes (and which of their chunks, times 256) that reach `least`, and those of which all is read
    uint16_t *const ones = reinterpret_cast<uint16_t *>(cand_v + kBuffer);
    uint8_t *const alls = reinterpret_cast<uint8_t *>(ones + 2 * blockDim.x);
    __shared__ int n_one, n_all, n_cand;
    __shared__ float sh_least;
    __shared__ int sh_kth;
    __shared__ Sums sh_sums[kScoreWarps];
    constexpr int V = Part<T>::kV, kPieces = 4;
    constexpr int kStep = 32 * kPieces;             // pieces per chunk
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int K = p.n_top, stride = p.splits * warps * kStep;
    pdl_trigger();
    pdl_wait();
    const Place<T> at(p, blockIdx.x);
    const int first = (at.split * warps + warp) * kStep;
    // chunks from in0 up to in1 lie within the row
    const int in0 = at.shift > 0 ? 1 : 0, in1 = (p.vocab + at.shift) / V - kStep;
    const uint4 *base = reinterpret_cast<const uint4 *>(at.x - at.shift) + lane;
    uint4 w[kPieces];
    auto edge = [&](int c) {            // (through a copy, which may lie in memory)
        uint4 t[kPieces];
        load_edge(at.x, at.shift, p.vocab, c + lane, t);
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            w[i] = t[i];
    };
    if (first < at.pieces) {
        if (first >= in0 && first <= in1) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                w[i] = __ldcs(base + first + 32 * i);
        } else {
            edge(first);
        }
    }
    const int given = p.token ? p.token[at.row] : -1;
    const bool has = given >= 0 && given < p.vocab;
    const float xg = has ? static_cast<float>(at.x[given]) : CUDART_NAN_F;
    // The tokens in front of the given one: up to its own piece those not below it, behind it
    // those above it. What its own piece has from it on is taken off again (with a given logit of
    // -inf that is also what lies beyond the row's ends, which counts as -inf).
    const int given_piece = RANK && has ? (given + at.shift) / V : -1;
    const float xa = RANK && has ? above(xg, T()) : CUDART_NAN_F;
    const int behind = given_piece * V - at.shift + lane;
    const bool counted = RANK && has && at.split == 0 && warp == 0 && lane < V && behind >= given;
    const float xb = counted && behind < p.vocab ? static_cast<float>(at.x[behind]) : -CUDART_INF_F;
    Part<T> part;
    Sums a = {-CUDART_INF_F, 0.f, 0.f, 0};
    float k1 = -CUDART_INF_F, k2 = k1, k3 = k1;
    uint32_t number = 0;
    for (int c = first; c < at.pieces; c += stride) {
        const float cm = Part<T>::highest(w);
        if (TOP) {
            const float k = fmaxf(Key<T>::of(cm, number), -CUDART_INF_F), less = fminf(k1, k);
            k3 = fmaxf(k3, fminf(k2, less));
            k2 = fmaxf(k2, less);
            k1 = fmaxf(k1, k);
            number = min(number + 1, Key<T>::kNumber);
        }
        if (RANK) {
            if (c <= given_piece && given_piece < c + kStep) {
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
                    part.count(w[i], c + 32 * i + lane <= given_piece ? xg : xa);
            } else {
                const float least = c <= given_piece ? xg : xa;
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
                    part.count(w[i], least);
            }
            part.settle();
        }
        // (masked tokens alone so far: they add nothing to any reference, and it stays -inf)
        const float up = fmaxf(a.R, cm * kLog2e4), rn = up == -CUDART_INF_F ? 0.f : up;
        const bool usual = fabsf(rn) < kLarge * kLog2e4;
        if (!usual) {
            uint4 copy[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                copy[i] = w[i];
            a = odd_chunk<T>(a, cm, copy);
        } else if (up > a.R) {
            const float d = 4.f * (a.R - up), f = ex2(d);
            if (ENT)                // (d may be beyond what 32 bits hold)
                a.t = f != 0.f ? (a.t + a.s * d) * f : 0.f;
            a.s *= f;
            a.R = up;
        }
        // each piece's successor is asked for when its tokens are in registers: 64 bytes a lane are on
        // their way (32 are too few to keep HBM busy)
        const int cn = c + stride;
        const bool inner = cn <= in1;
        const uint64_t c2 = pack2(kLog2e, kLog2e), r2 = pack2(-4.f * rn, -4.f * rn);
        const typename Part<T>::Low low(usual ? rn : 0.f);
        uint64_t acc = 0, ent = 0;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const uint4 x = w[i];
            if (inner)
                w[i] = __ldcs(base + cn + 32 * i);
            Part<T>::template terms<ENT>(x, low, c2, r2, acc, ent);
        }
        if (usual) {
            const float2 s2 = unpack2(acc);
            a.s += s2.x + s2.y;
            if (ENT) {
                const float2 t2 = unpack2(ent);
                a.t += t2.x + t2.y;
            }
        }
        if (!inner && cn < at.pieces)
            edge(cn);
    }
    if (RANK)
        a.front = part.counted() - (counted && xb == xg ? 1 : 0) -
                  (has && xg == -CUDART_INF_F && at.split == 0 && tid == 0 ? at.shift : 0);
    // the sums of the warp, of the CTA
    auto warp_join = [&](const Sums &v) {
        Sums o = moved<ENT>(v, unorder(__reduce_max_sync(kAll, order(v.R))));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            o.s += __shfl_xor_sync(kAll, o.s, d);
            if (ENT)
                o.t += __shfl_xor_sync(kAll, o.t, d);
        }
        o.front = RANK ? __reduce_add_sync(kAll, v.front) : 0;
        return o;
    };
    const Sums none = {-CUDART_INF_F, 0.f, 0.f, 0};
    a = warp_join(a);
    if (lane == 0)
        sh_sums[warp] = a;
    Best best;
    best.clear();
    if (TOP) {
        lane_k[tid] = k1;
        lane_k[tid + blockDim.x] = k2;
        lane_k[tid + 2 * blockDim.x] = k3;
    }
    if (TOP && tid == 0)
        sh_kth = INT_MAX;
    __syncthreads();
    if (TOP) {
        // the K-th highest key: of many by counting, in every lane, the keys above its own, of a few by
        // taking the highest out, one after the other (6 us more of 126 for 8192 rows with 20
        // tokens, 2 of 14 for one row with 32)
        const bool many = K > 2 * warps;
        if (many) {
            int before = 0;
            for (int i = 0; i < 8 * warps; ++i) {
                const float4 q = reinterpret_cast<const float4 *>(lane_k)[i];
                before += (q.x > k1) + (q.y > k1) + (q.z > k1) + (q.w > k1);
            }
            const int low = __reduce_min_sync(kAll, before < K ? order(k1) : INT_MAX);
            if (lane == 0 && low != INT_MAX)
                atomicMin(&sh_kth, low);
            __syncthreads();
        }
        if (warp == 0) {
            float least = -CUDART_INF_F;
            if (many) {
                least = unorder(sh_kth);
            } else {
                float h[kScoreWarps], hm = -CUDART_INF_F;
#pragma unroll
                for (int i = 0; i < kScoreWarps; ++i) {
                    h[i] = i < warps ? lane_k[32 * i + lane] : -CUDART_INF_F;
                    hm = fmaxf(hm, h[i]);
                }
                int left = K;
                while (left > 0) {          // the highest are taken out, one of each lane that holds it
                    least = unorder(__reduce_max_sync(kAll, order(hm)));
                    if (least == -CUDART_INF_F)
                        break;
                    const bool mine = hm == least;
                    left -= __popc(__ballot_sync(kAll, mine));
                    float rest = -CUDART_INF_F;
                    bool out = !mine;
#pragma unroll
                    for (int i = 0; i < kScoreWarps; ++i) {
                        if (i >= warps)
                            break;
                        const bool hit = !out && h[i] == least;
                        h[i] = hit ? -CUDART_INF_F : h[i];
                        out = out || hit;
                        rest = fmaxf(rest, h[i]);
                    }
                    hm = rest;
                }
            }
            // (fewer than K lanes have a token that is not masked: all such tokens, and the lowest masked
            // ones behind them)
            least = least == -CUDART_INF_F ? -FLT_MAX : Key<T>::lo(least);
            int n1 = 0, n2 = 0;
            for (int i = 0; i < warps; ++i) {
                const int l = 32 * i + lane;
                const float q1 = lane_k[l], q2 = lane_k[l + blockDim.x], q3 = lane_k[l + 2 * blockDim.x];
                const bool in1 = Key<T>::hi(q1) >= least, in2 = Key<T>::hi(q2) >= least;
                const bool all = Key<T>::hi(q3) >= least || (in1 && Key<T>::number(q1) == Key<T>::kNumber) ||
                                 (in2 && Key<T>::number(q2) == Key<T>::kNumber);
                const uint32_t b1 = __ballot_sync(kAll, in1 && !all), b2 = __ballot_sync(kAll, in2 && !all);
                const uint32_t b3 = __ballot_sync(kAll, all), before = (1u << lane) - 1u;
                if (in1 && !all)
                    ones[n1 + __popc(b1 & before)] = static_cast<uint16_t>(l);
                n1 += __popc(b1);
                if (in2 && !all)
                    ones[n1 + __popc(b2 & before)] = static_cast<uint16_t>(l + 256);
                n1 += __popc(b2);
                if (all)
                    alls[n2 + __popc(b3 & before)] = static_cast<uint8_t>(l);
                n2 += __popc(b3);
            }
            if (lane == 0) {
                n_one = n1;
                n_all = n2;
                n_cand = 0;
                sh_least = least;
            }
        }
        __syncthreads();
        const float least = sh_least;
        const int begun = at.split * warps * kStep, mid = n_one * kPieces;
        const int rounds = at.pieces > begun ? (at.pieces - begun + stride - 1) / stride : 0;
        const int total = mid + n_all * rounds * kPieces;
        // (the first warp looks through as many pieces by itself as surely fit the buffer)
        const bool alone = total * V <= kBuffer;
        const int step = alone ? 32 : blockDim.x;
        constexpr int kU = 2;           // pieces of a thread on their way at once
        int found = 0;
        for (int i0 = warp * 32; i0 < total && (!alone || warp == 0); i0 += kU * step) {
            uint4 word[kU];
            int piece[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int i = i0 + u * step + lane;
                piece[u] = at.pieces;       // (nothing)
                if (i < mid) {
                    const int l = ones[i / kPieces], which = l >> 8;
                    const int r = Key<T>::number(lane_k[(l & 255) + which * blockDim.x]);
                    piece[u] = begun + (l >> 5 & 7) * kStep + r * stride + 32 * (i % kPieces) + (l & 31);
                } else if (i < total) {
                    const int k = i - mid, r = k / n_all, l = alls[k - r * n_all];
                    piece[u] = begun + (l >> 5) * kStep + (r / kPieces) * stride + 32 * (r % kPieces) + (l & 31);
                }
                load_pieces<T, 1>(at.x, at.shift, p.vocab, min(piece[u], at.pieces), word + u);
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                float x[V];
                Chunk<T>::unpack(word[u], x);
                uint32_t hits = 0;
#pragma unroll
                for (int j = 0; j < V; ++j)     // (what lies beyond the row's ends is -inf)
                    hits |= x[j] >= least ? 1u << j : 0u;
                uint32_t some;
                while ((some = __ballot_sync(kAll, hits != 0)) != 0) {
                    int base = found;
                    if (!alone) {
                        if (lane == 0)
                            base = atomicAdd(&n_cand, __popc(some));
                        base = __shfl_sync(kAll, base, 0);
                    }
                    found += __popc(some);
                    const int j = __ffs(hits) - 1, v = piece[u] * V - at.shift + j;
                    float xj = -CUDART_INF_F;
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        xj = i == j ? x[i] : xj;
                    const int to = hits ? base + __popc(some & ((1u << lane) - 1u)) : -1;
                    hits &= hits - 1;
                    if (to >= 0 && to < kBuffer) {
                        cand_x[to] = xj;
                        cand_v[to] = v;
                    }
                    // (many equal logits, or many high ones in few lanes)
                    if (__any_sync(kAll, to >= kBuffer))
                        best.offer(xj, to >= kBuffer ? v : -1, K, lane);
                }
            }
        }
        if (alone) {
            if (tid == 0)
                n_cand = found;
        } else {
            __syncthreads();
            if (n_cand > kBuffer) {
                if (lane < K) {
                    sh_x[lane * warps + warp] = best.x;
                    sh_v[lane * warps + warp] = best.v;
                }
                __syncthreads();
            }
        }
    }
    if (warp != 0)
        return;
    __syncwarp();
    if (TOP) {
        const int n = n_cand;
        if (n <= 64) {
            best = placed(cand_x, cand_v, n, K, lane, sh_x, sh_v);
        } else {
            best.clear();       // (its own list is among the others)
            if (n > kBuffer)
                best = merged(best, sh_x, sh_v, K * warps, K, lane);
            best = merged(best, cand_x, cand_v, min(n, kBuffer), K, lane);
        }
        if (sh_least == -FLT_MAX) {
            const int piece = at.split * warps * kStep;
            for (int v0 = max(piece * V - at.shift, 0); v0 < p.vocab && best.tv < 0; v0 += 32) {
                const int v = v0 + lane;
                const bool own = v < p.vocab && (v + at.shift) / V / (warps * kStep) % p.splits == at.split;
                const bool masked = own && static_cast<float>(at.x[v]) == -CUDART_INF_F;
                best.offer(-CUDART_INF_F, masked ? v : -1, K, lane);
            }
        }
    }
    if (warps > 1)
        a = warp_join(lane < warps ? sh_sums[lane] : none);
    if (p.splits > 1) {
        const size_t parts = static_cast<size_t>(at.row) * p.splits;
        if (lane == 0)
            p.part[parts + at.split] = make_float4(a.R, a.s, a.t, __int_as_float(a.front));
        if (TOP && lane < K) {
            const size_t to = parts * K + static_cast<size_t>(lane) * p.splits + at.split;
            p.part_x[to] = best.x;
            p.part_v[to] = best.v;
        }
        __threadfence();
        __syncwarp();
        int last = 0;
        if (lane == 0)
            last = atomic_add_acq_rel_gpu(p.tickets + at.row, 1) == p.splits - 1;
        if (!__shfl_sync(kAll, last, 0))
            return;
        __threadfence();
        if (lane == 0)
            p.tickets[at.row] = 0;
        a = none;
        for (int i = lane; i < p.splits; i += 32) {
            const float4 v = __ldcg(p.part + parts + i);
            const Sums b = {v.x, v.y, v.z, __float_as_int(v.w)};
            const float R = fmaxf(a.R, b.R);
            const Sums x = moved<ENT>(a, R), y = moved<ENT>(b, R);
            a = Sums{R, x.s + y.s, x.t + y.t, x.front + y.front};
        }
        a = warp_join(a);
        if (TOP) {
            best.clear();
            best = merged(best, p.part_x + parts * K, p.part_v + parts * K, K * p.splits, K, lane);
        }
    }
    const float ls = logf(a.s);
    const bool sound = isfinite(a.R) && isfinite(ls);
    // lse less ln s is 4 R / log2 e, as ref + rest: in fp32 alone it would round at the size of the
    // logits (and the few units for 64 bits would hold up short rows: 8192 of 1000 tokens 22.5 us then).
    // From kLarge on the reference is half the largest logit.
    constexpr double kPerR = 1. / kLog2e4;
    constexpr float kPer = static_cast<float>(kPerR), kPerRest = static_cast<float>(kPerR - kPer);
    const bool small = fabsf(a.R) < kLarge * kLog2e4;
    const float ref = small ? __fmul_rn(a.R, kPer) : 2.f * a.R;
    const float rest = small ? fmaf(a.R, kPer, -ref) + a.R * kPerRest : 0.f;
    // (x - ref exactly, as d + lost; a probability is at most 1 and entropy at least 0, whatever the
    // roundings say)
    auto log_p = [&](float x) {
        const float d = x - ref, b = d - x, lost = (x - (d - b)) - (ref + b);
        const float l = (d - ls) + (fabsf(d) < CUDART_INF_F ? lost - rest : 0.f);
        return sound ? fminf(l, 0.f) : CUDART_NAN_F;
    };
    if (lane == 0) {
        if (p.logprob)
            p.logprob[at.row] = given < 0 ? 0.f : has ? log_p(xg) : CUDART_NAN_F;
        if (RANK)
            p.rank[at.row] = has && sound ? a.front : -1;
        if (ENT)
            p.entropy[at.row] = sound ? fmaxf(ls - a.t / a.s * CUDART_LN2_F, 0.f) : CUDART_NAN_F;
    }
    if (TOP && lane < K) {
        const size_t to = static_cast<size_t>(at.row) * K + lane;
        p.top_token[to] = sound ? best.v : -1;
        p.top_logprob[to] = log_p(best.x);
    }
}

template <typename T, bool TOP>
cudaError_t launch_top(const ScoreParams &p, cudaStream_t stream)
{
    const dim3 grid(p.n_rows * p.splits), block(32 * p.warps);
    const size_t sh = TOP ? 32 * p.warps * (3 * sizeof(float) + 2 * sizeof(uint16_t) + 1) + 2 * kBuffer * sizeof(float) : 0;
    if (p.rank)
        return p.entropy ? launch_pdl(score_kernel<T, TOP, true, true>, grid, block, sh, stream, p)
                         : launch_pdl(score_kernel<T, TOP, true, false>, grid, block, sh, stream, p);
    return p.entropy ? launch_pdl(score_kernel<T, TOP, false, true>, grid, block, sh, stream, p)
                     : launch_pdl(score_kernel<T, TOP, false, false>, grid, block, sh, stream, p);
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
