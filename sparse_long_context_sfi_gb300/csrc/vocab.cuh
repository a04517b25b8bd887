// vocab.cuh -- one pass over the logits of a row by the warps of a CTA, for beam.cu and score.cu: chunks in
// registers (of beam.cu 512 tokens; of score.cu 64 bytes a lane, 512 of fp32 and 1024 of bf16), references
// that keep the sums of exponentials in range, and the sorted list of a warp's best tokens.
#pragma once

#include "sfi_device.cuh"

#include <math_constants.h>

namespace sfi {
namespace {

constexpr int kLaneTok = 16;                 // tokens per lane and chunk
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLarge = 0x1p29f;            // logits of this size and beyond: see reference()
constexpr float kLog2e4 = 0.25f * kLog2e;

// What a logit is measured from, in units of 2^4 (by which exp(x) is 2^(x log2 e - 4 R)). Below
// kLarge R = fl(x log2 e) / 4; x log2 e is off from it by 2^5 at most, so that the power stays in
// range. From kLarge on two different logits are at least 64 apart, and in a row's sum only those
// equal to the largest are left (the next has e^-64 of its weight or less): there it is enough that
// R = x / 2 is exact, and above (or, negative, below) all the others.
__device__ __forceinline__ float reference(float x)
{
    return fabsf(x) < kLarge ? x * kLog2e4 : 0.5f * x;
}

// a before b: higher logit, then lower token (empty places, v < 0, last)
__device__ __forceinline__ bool better(float xa, int va, float xb, int vb)
{
    // (unsigned: an empty place, -1, is behind every token)
    return xa > xb || (xa == xb && static_cast<uint32_t>(va) < static_cast<uint32_t>(vb));
}

// Two floats at a time (sm_100 has packed fp32 adds and multiply-adds).
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

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a term relative to reference a counts relative to b.
__device__ __forceinline__ float apart(float a, float b) { return ex2(4.f * (a - b)); }

// An integer that orders like the float (and back), for the warp's integer reductions.
__device__ __forceinline__ int order(float x)
{
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}

__device__ __forceinline__ float unorder(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// The warp's K best so far: lane j holds the j-th, lanes from K on hold nothing.
struct Best {
    float x;
    int v;
    float tx;      // the last of them (every lane): what a token has to beat
    int tv;

    __device__ __forceinline__ void clear()
    {
        x = tx = -CUDART_INF_F;
        v = tv = -1;
    }
    // every lane calls it with the same (cx, cv), better than (tx, tv)
    __device__ __forceinline__ void insert(float cx, int cv, int K, int lane)
    {
        const uint32_t m = __ballot_sync(kAll, better(cx, cv, x, v));
        const int pos = __ffs(m) - 1;
        const float ux = __shfl_up_sync(kAll, x, 1);
        const int uv = __shfl_up_sync(kAll, v, 1);
        if (lane >= pos && lane < K) {
            x = lane == pos ? cx : ux;
            v = lane == pos ? cv : uv;
        }
        tx = __shfl_sync(kAll, x, K - 1);
        tv = __shfl_sync(kAll, v, K - 1);
    }
    // each lane offers one candidate (v < 0: none); from the last lane down
    __device__ __forceinline__ void offer(float cx, int cv, int K, int lane)
    {
        uint32_t m = __ballot_sync(kAll, cv >= 0 && better(cx, cv, tx, tv));
        while (m) {
            const int src = 31 - __clz(m);
            insert(__shfl_sync(kAll, cx, src), __shfl_sync(kAll, cv, src), K, lane);
            m = __ballot_sync(kAll, cv >= 0 && better(cx, cv, tx, tv)) & ((1u << src) - 1u);
        }
    }
    // the first candidates, one per lane: sorted over the warp (bitonic), the first K kept
    __device__ __forceinline__ void start(float cx, int cv, int K, int lane)
    {
        x = cv >= 0 ? cx : -CUDART_INF_F;
        v = cv;
#pragma unroll
        for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
            for (int d = size >> 1; d > 0; d >>= 1) {
                const float ox = __shfl_xor_sync(kAll, x, d);
                const int ov = __shfl_xor_sync(kAll, v, d);
                // descending runs where the size's bit of the lane is clear
                const bool first = ((lane & d) == 0) == ((lane & size) == 0);
                if (better(ox, ov, x, v) == first) {
                    x = ox;
                    v = ov;
                }
            }
        }
        if (lane >= K) {
            x = -CUDART_INF_F;
            v = -1;
        }
        tx = __shfl_sync(kAll, x, K - 1);
        tv = __shfl_sync(kAll, v, K - 1);
    }
};

// 16 tokens of one lane: V = 16 / sizeof(T) of them per 16-byte piece, pieces 32 lanes apart.
template <typename T>
struct Chunk;

template <>
struct Chunk<float> {
    static constexpr int kV = 4;
    static __device__ __forceinline__ void unpack(const uint4 &w, float *x)
    {
        x[0] = __uint_as_float(w.x);
        x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z);
        x[3] = __uint_as_float(w.w);
    }
};

template <>
struct Chunk<__nv_bfloat16> {
    static constexpr int kV = 8;
    static __device__ __forceinline__ void unpack(const uint4 &w, float *x)
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
};

// The pieces of this lane in the chunk that begins with piece0; those that reach over either end of the
// row are put together from its tokens (others: -inf, which no sum and no list sees). (256 rows of 128001
// tokens take a selection 31.9 us, with score.cu's load_pieces in its place 32.2.)
template <typename T>
__device__ __forceinline__ void load_chunk(const T *row, int shift, int vocab, int piece0, int lane,
                                           uint4 *w)
{
    constexpr int V = Chunk<T>::kV;
#pragma unroll
    for (int i = 0; i < kLaneTok / V; ++i) {
        const int at = (piece0 + 32 * i + lane) * V - shift;   // first token of the piece
        if (at >= 0 && at + V <= vocab) {
            w[i] = __ldcs(reinterpret_cast<const uint4 *>(row + at));
        } else {
            T t[V];
#pragma unroll
            for (int j = 0; j < V; ++j)
                t[j] = at + j >= 0 && at + j < vocab ? row[at + j] : static_cast<T>(-CUDART_INF_F);
            w[i] = *reinterpret_cast<const uint4 *>(t);
        }
    }
}

}  // namespace
}  // namespace sfi
