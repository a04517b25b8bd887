// chunk.cuh -- which rows of a packed chunk belong to which sequence, and their places in the cache.
#pragma once

#include "sfi_device.cuh"

namespace sfi {

// What a call asks of a sequence beside sound rows: nothing, a length within max_len, room for the
// rows, too.
enum { kNeedRows = 0, kNeedLength = 1, kNeedRoom = 2 };

// Whether sequence b's chunk is sound: rows within bounds and no other's, room in the cache. A
// warp call, every lane the same b. Where the starts run backwards somewhere, rows belong to the
// first sequence that claims them: one that begins before an earlier start is left out.
template <int NEED = kNeedRoom>
__device__ __forceinline__ bool chunk_ok(const ChunkParams &p, int b, int lane, int &r0, int &n, int &L,
                                         bool report)
{
    r0 = p.row_start ? p.row_start[b] : b;
    const int r1 = p.row_start ? p.row_start[b + 1] : b + 1;
    n = r1 - r0;
    L = p.pg.seq_len[b];
    bool owned = true;
    if (p.row_start)
        for (int i = lane; i < b; i += 32)
            owned = owned && p.row_start[i] <= r0;
    owned = __all_sync(0xffffffffu, owned) != 0;
    uint32_t bad = 0;
    if (r0 < 0 || n < 0 || r1 > p.n_rows || n > p.max_rows || (n > 0 && !owned))
        bad = 0x20u;  // SFI_DEVERR_ROWS
    else if (NEED >= kNeedLength && (L < 0 || L > p.pg.max_len))
        bad = 0x8u;   // SFI_DEVERR_LENGTH
    else if (NEED >= kNeedRoom && n > p.pg.capacity - L)
        bad = 0x2u;   // SFI_DEVERR_CAPACITY
    if (bad && report)
        raise_error(p.pg.err, bad);
    return bad == 0;
}

// The sequence and the position of packed row r, -1 where the row is not served. One warp, every
// lane the same r: the row's sequence is the one before the first start behind r, found
// in one round trip (a sound sequence's own rows are in front of every later start that counts).
template <int NEED = kNeedRoom>
__device__ __forceinline__ int chunk_seq(const ChunkParams &p, int r, int lane, int &pos)
{
    int b = r;
    if (r >= p.n_rows)
        return -1;
    if (p.row_start) {
        int behind = p.pg.batch + 1;
        for (int i = lane; i <= p.pg.batch; i += 32)
            if (p.row_start[i] > r)
                behind = min(behind, i);
        b = __reduce_min_sync(0xffffffffu, behind) - 1;
        if (b < 0 || b >= p.pg.batch)
            return -1;
    }
    int s0, n, L;
    if ((p.pg.active && !p.pg.active[b]) || !chunk_ok<NEED>(p, b, lane, s0, n, L, false) || r < s0 || r >= s0 + n)
        return -1;
    pos = L + r - s0;
    return b;
}

// The cache row of (layer 0, head 0) for position pos of sequence b, -1 where it has no page.
__device__ __forceinline__ long long cache_row(const PageParams &p, int b, int pos)
{
    if (p.page_size == 0)
        return static_cast<long long>(b) * p.n_kv_heads * p.capacity + pos;
    const int page = p.table[static_cast<size_t>(b) * p.max_pages + (pos >> 4)];
    if (page < 0 || page >= p.n_pages)
        return -1;
    return static_cast<long long>(page) * p.n_kv_heads * 16 + (pos & 15);
}

// The same for packed row r (a warp call).
__device__ __forceinline__ long long chunk_dst(const ChunkParams &p, int r, int lane)
{
    int pos;
    const int b = chunk_seq(p, r, lane, pos);
    return b < 0 ? -1 : cache_row(p.pg, b, pos);
}

// The lengths after the rows of a chunk, by one block: a warp per sequence, which first looks over
// the chunk's pages.
__device__ __forceinline__ void advance_lengths(const ChunkParams &p)
{
    const int lane = threadIdx.x & 31;
    for (int b = threadIdx.x >> 5; b < p.pg.batch; b += static_cast<int>(blockDim.x >> 5)) {
        if (p.pg.active && !p.pg.active[b])
            continue;
        int s0, n, L;
        if (!chunk_ok(p, b, lane, s0, n, L, lane == 0))
            continue;
        bool good = true;
        if (p.pg.page_size != 0 && n > 0) {
            for (int c = (L >> 4) + lane; c <= (L + n - 1) >> 4; c += 32) {
                const int e = p.pg.table[static_cast<size_t>(b) * p.pg.max_pages + c];
                good = good && e >= 0 && e < p.pg.n_pages;
            }
        }
        good = __all_sync(0xffffffffu, good);
        __syncwarp();
        if (lane == 0) {
            if (good)
                p.pg.seq_len[b] = L + n;
            else
                raise_error(p.pg.err, 0x1u);  // SFI_DEVERR_PAGE_RANGE
        }
    }
}

}  // namespace sfi
