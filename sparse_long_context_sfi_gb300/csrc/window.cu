// window.cu -- attention of a chunk of rows under sinks and a sliding window, straight from
// the cache: one warp per (row, query head), online softmax over the visible positions.
#include "sfi_device.cuh"

#include <math_constants.h>

namespace sfi {
namespace {

__global__ void __launch_bounds__(256) window_simple_kernel(const WindowParams p)
{
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int hq = p.n_kv_heads * p.group;
    const long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (w >= static_cast<long long>(p.n_layers) * p.n_rows * hq)
        return;
    const int h = static_cast<int>(w % hq);
    const long long lr = w / hq;
    const int r = static_cast<int>(lr % p.n_rows), layer = static_cast<int>(lr / p.n_rows);
    int b = r;
    if (p.row_start) {
        if (r < p.row_start[0] || r >= p.row_start[p.batch])
            return;
        int lo = 0, hi = p.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.row_start[mid] <= r)
                lo = mid;
            else
                hi = mid;
        }
        b = lo;
    }
    if (p.active && !p.active[b])
        return;
    const int s0 = p.row_start ? p.row_start[b] : b, s1 = p.row_start ? p.row_start[b + 1] : b + 1;
    const int L = p.seq_len[b], n = s1 - s0;
    uint32_t bad = 0;
    if (n < 0 || s0 < 0 || s1 > p.n_rows || n > p.max_rows || r < s0 || r >= s1)
        bad = 0x20u;  // SFI_DEVERR_ROWS
    else if (L < n || L > p.max_len)
        bad = 0x8u;   // SFI_DEVERR_LENGTH
    if (bad) {
        if (lane == 0)
            raise_error(p.err, bad);
        return;
    }
    const int pos = L - n + (r - s0);
    const int low = max(0, pos - p.n_window + 1), ns = min(p.n_sink, low);
    const uint2 *q = static_cast<const uint2 *>(p.q) + w * 32 + lane;
    const float2 q01 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&q->x));
    const float2 q23 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&q->y));
    float m = -CUDART_INF_F, l = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
    const int total = ns + pos - low + 1, kvh = h / p.group;
    for (int i = 0; i < total; ++i) {
        const int j = i < ns ? i : low + i - ns;
        long long row;
        if (p.page_size == 0) {
            row = (static_cast<long long>(layer * p.batch + b) * p.n_kv_heads + kvh) * p.capacity + j;
        } else {
            const int page = p.page_table[static_cast<size_t>(b) * p.max_pages + (j >> 4)];
            if (page < 0 || page >= p.n_pages) {
                if (lane == 0)
                    raise_error(p.err, 0x1u);  // SFI_DEVERR_PAGE_RANGE
                continue;
            }
            row = (static_cast<long long>(layer * p.n_pages + page) * p.n_kv_heads + kvh) * 16 + (j & 15);
        }
        const uint2 kx = static_cast<const uint2 *>(p.k)[row * 32 + lane];
        const uint2 vx = static_cast<const uint2 *>(p.v)[row * 32 + lane];
        const float2 k01 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&kx.x));
        const float2 k23 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&kx.y));
        const float2 v01 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&vx.x));
        const float2 v23 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&vx.y));
        float z = q01.x * k01.x + q01.y * k01.y + q23.x * k23.x + q23.y * k23.y;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            z += __shfl_xor_sync(0xffffffffu, z, d);
        z *= 0.08838834764831845f;   // 1 / sqrt(128)
        const float mn = fmaxf(m, z), a = expf(m - mn), e = expf(z - mn);
        m = mn;
        l = l * a + e;
        o0 = o0 * a + e * v01.x;
        o1 = o1 * a + e * v01.y;
        o2 = o2 * a + e * v23.x;
        o3 = o3 * a + e * v23.y;
    }
    const float inv = 1.f / l;
    const size_t at = static_cast<size_t>(w) * 128 + lane * 4;
    if (p.out_fp32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) =
            make_float4(o0 * inv, o1 * inv, o2 * inv, o3 * inv);
    } else {
        __nv_bfloat162 *o = reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(p.out) + at);
        o[0] = __floats2bfloat162_rn(o0 * inv, o1 * inv);
        o[1] = __floats2bfloat162_rn(o2 * inv, o3 * inv);
    }
}

}  // namespace

cudaError_t launch_window(const WindowParams &p, cudaStream_t stream)
{
    const long long warps = static_cast<long long>(p.n_layers) * p.n_rows * p.n_kv_heads * p.group;
    const cudaError_t e = launch_pdl(window_simple_kernel, dim3(static_cast<unsigned>((warps + 7) / 8)),
                                     dim3(256), 0, stream, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sfi
