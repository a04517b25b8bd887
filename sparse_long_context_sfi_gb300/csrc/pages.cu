// pages.cu -- upkeep of a paged KV cache on the device (page tables and reference counts), the
// rows of a prompt chunk, and the reordering of whole sequences.
//
// Integer bookkeeping is done by one CTA per call where it needs an order (lowest free page
// first), so that the result never depends on timing; everything that moves K and V bytes
// runs on the whole GPU. A page of one layer and tensor is n_kv_heads * 4 KB, contiguous.
//
// Measured (GB300, copy rate 6.78 TB/s): rows of four 8K chunks 38 us (7.0 TB/s of read and
// written bytes), a quarter of a 16K-page pool moved in 77 us (7.0 TB/s); 8 sequences with
// their packed memory (31 MB) forked to 24 others in 27.7 us with tables and counts (29.4 when each
// copy read its source); 8 sequences of 4096 contiguous rows (134 MB) forked to 24 others in 89 us
// (6.0 TB/s), all 32 moved in 167 (6.4); the one-CTA plans take 5 to 8 us, round trips to L2.
//
// Kernels here that write what a fast step may read before its own wait (packed memory, `ok`
// masks) let no dependent start early; the others start theirs at entry.
#include "chunk.cuh"
#include "sfi_device.cuh"

namespace sfi {
namespace {

constexpr int kPlanThreads = 1024;
constexpr uint32_t kFull = 0xffffffffu;

// ------------------------------------------------------------------- release and eviction

// Drops the references of the entries in columns [c0, c1) of each active sequence: all of them
// (release) or the pages wholly between the sinks and the window (evict). Latency-bound: a
// table row is a few KB.
__global__ void __launch_bounds__(256) drop_pages_kernel(const PageParams p, int evict, int n_sink,
                                                         int n_window)
{
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.y;
    if (p.active && !p.active[b])
        return;
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (!evict && blockIdx.x == 0 && threadIdx.x == 0)
        p.seq_len[b] = 0;
    int c0 = 0, c1 = p.max_pages;
    if (evict) {
        const int dead = p.seq_len[b] - n_window;   // positions below it are out of the window
        c0 = n_sink / 16 + (n_sink % 16 != 0);
        c1 = dead > 0 ? min(dead / 16, p.max_pages) : 0;
    }
    if (c < c0 || c >= c1)
        return;
    int32_t *e = p.table + static_cast<size_t>(b) * p.max_pages + c;
    const int page = *e;
    if (page < 0)
        return;
    *e = -1;
    if (page >= p.n_pages) {
        raise_error(p.err, 0x1u);  // SFI_DEVERR_PAGE_RANGE
    } else if (atomicSub(p.refs + page, 1) <= 0) {
        atomicAdd(p.refs + page, 1);
        raise_error(p.err, 0x80u);  // SFI_DEVERR_REFS
    }
}

// ------------------------------------------------------------------------------- reserving

// Sum over the block's 32 warps of `v` (one value per warp, from lane 0), as an exclusive
// prefix per warp and the total; every thread calls it.
__device__ __forceinline__ int warp_prefix(int v, int *sh, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0)
        sh[warp] = v;
    __syncthreads();
    int x = sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o)
            x += y;
    }
    total = __shfl_sync(kFull, x, 31);
    const int mine = __shfl_sync(kFull, x, warp) - v;
    __syncthreads();
    return mine;
}

// Inclusive prefix sums over the warp.
__device__ __forceinline__ int warp_scan(int x)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o)
            x += y;
    }
    return x;
}

// One CTA. A task is 32 columns of one sequence's range; tasks are numbered by sequence, then
// position, so that the running count of entries that need a page, over tasks, is the order in
// which pages are handed out. (A) a warp per task marks its entries, four tasks in flight;
// (B) the marks are counted; (C) the lowest free pages are listed; (D) a warp per task hands
// them out. The marks are kept because the sharing rule of (A) reads other sequences' entries,
// which (D) changes. What is left is latency: about eight dependent round trips to L2.
constexpr int kTasksInSmem = 1024, kListInSmem = 2048;

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const PageParams p,
                                                               const int32_t *n_new, uint8_t *ok,
                                                               const PageScratch s)
{
    __shared__ int first[kMaxBatch], last[kMaxBatch], task0[kMaxBatch + 1];
    __shared__ int lean[kMaxBatch];         // the last sequence that has to leave a page for this one
    __shared__ int8_t state[kMaxBatch];     // 0: to be served, -1: refused or not active
    __shared__ uint8_t tail[kMaxBatch];     // rows in the current page
    __shared__ uint32_t sh_marks[kTasksInSmem];
    __shared__ int sh_count[kTasksInSmem + 1], sh_list[kListInSmem], sh[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    // the first chunk's counts are asked for at once: nothing before (D) changes them
    int held[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        held[i] = warp * 512 + lane + 32 * i < p.n_pages ? p.refs[warp * 512 + lane + 32 * i] : 1;
    if (tid < p.batch) {
        const int b = tid;
        const bool on = !p.active || p.active[b];
        const int L = p.seq_len[b], n = n_new ? n_new[b] : 1;
        int f = 0, l = -1, st = on ? 0 : -1;
        if (on && (L < 0 || L > p.max_len)) {
            raise_error(p.err, 0x8u);  // SFI_DEVERR_LENGTH
            st = -1;
        } else if (on && n > 0) {
            if (n > p.capacity - L) {
                raise_error(p.err, 0x2u);  // SFI_DEVERR_CAPACITY
                st = -1;
            } else {
                f = L >> 4;
                l = (L + n - 1) >> 4;
            }
        }
        first[b] = f;
        last[b] = l;
        lean[b] = -1;
        tail[b] = static_cast<uint8_t>(L & 15);
        state[b] = static_cast<int8_t>(st);
        s.copies[b] = make_int4(0, 0, 0, 0);    // page to, page from, rows
    }
    __syncthreads();
    if (warp == 0) {
        int run = 0;
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
            const int b = b0 + lane;
            const int v = b < p.batch && last[b] >= first[b] ? ((last[b] - first[b]) >> 5) + 1 : 0;
            const int x = warp_scan(v);
            if (b < p.batch)
                task0[b] = run + x - v;
            run += __shfl_sync(kFull, x, 31);
        }
        if (lane == 0)
            task0[p.batch] = run;
    }
    __syncthreads();
    const int tasks = task0[p.batch];
    uint32_t *marks = tasks <= kTasksInSmem ? sh_marks : s.marks;
    int *count = tasks <= kTasksInSmem ? sh_count : s.counts;
    // the sequence of a task: the last b with task0[b] <= t
    auto owner = [&](int t) {
        int lo = 0, hi = p.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (task0[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        return lo;
    };
    // (A)
    for (int t0 = warp; t0 < tasks; t0 += 128) {      // tasks t0, t0 + 32, t0 + 64, t0 + 96
        int b[4], c0[4], e[4], holders[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            b[q] = t0 + 32 * q < tasks ? owner(t0 + 32 * q) : -1;
            c0[q] = b[q] < 0 ? 0 : first[b[q]] + 32 * (t0 + 32 * q - task0[b[q]]);
            e[q] = b[q] >= 0 && c0[q] + lane <= last[b[q]]
                       ? p.table[static_cast<size_t>(b[q]) * p.max_pages + c0[q] + lane]
                       : 0x7fffffff;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            holders[q] = e[q] >= 0 && e[q] < p.n_pages ? p.refs[e[q]] : 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (b[q] < 0)
                continue;
            const bool in = c0[q] + lane <= last[b[q]];
            bool want = in && (e[q] < 0 || e[q] >= p.n_pages);   // (a bad entry ahead is replaced)
            if (in && e[q] >= p.n_pages)
                raise_error(p.err, 0x1u);
            // shared pages (as a rule one per sequence, its current page): the warp counts the
            // earlier sequences that reserve on the same page (and whose current page is there)
            for (uint32_t sm = __ballot_sync(kFull, holders[q] > 1); sm != 0; sm &= sm - 1) {
                const int src = __ffs(sm) - 1, page = __shfl_sync(kFull, e[q], src), col = c0[q] + src;
                int before = 0, leaver = -1;
                for (int o = lane; o < b[q]; o += 32) {
                    const int32_t *row = p.table + static_cast<size_t>(o) * p.max_pages;
                    if (col >= first[o] && col <= last[o] && row[col] == page &&
                        (col == first[o] || !tail[o] || (row[first[o]] >= 0 && row[first[o]] < p.n_pages))) {
                        ++before;
                        leaver = o;
                    }
                }
                before = __reduce_add_sync(kFull, before);
                leaver = __reduce_max_sync(kFull, leaver);
                if (lane == src) {
                    want = holders[q] - before > 1;
                    if (!want)
                        atomicMax(lean + b[q], leaver);
                }
            }
            const uint32_t m = __ballot_sync(kFull, want);
            if (lane == 0) {
                marks[t0 + 32 * q] = m;
                // a current page that holds rows has to be there
                if (c0[q] == first[b[q]] && tail[b[q]] && (e[q] < 0 || e[q] >= p.n_pages)) {
                    raise_error(p.err, 0x1u);  // SFI_DEVERR_PAGE_RANGE
                    state[b[q]] = -1;
                }
            }
        }
    }
    __syncthreads();
    // (B)
    int total = 0;
    for (int t0 = 0; t0 < tasks; t0 += kPlanThreads) {
        const int t = t0 + tid;
        int v = 0;
        if (t < tasks) {
            if (state[owner(t)] != 0)
                marks[t] = 0;       // refused: nothing is handed out
            v = __popc(marks[t]);
        }
        const int x = warp_scan(v);
        int sum;
        const int before = warp_prefix(__shfl_sync(kFull, x, 31), sh, sum);
        if (t < tasks)
            count[t] = total + before + x - v;
        total += sum;
    }
    if (tid == 0)
        count[tasks] = total;
    int32_t *list = total <= kListInSmem ? sh_list : s.list;
    // (C) each warp takes 512 consecutive pages of a chunk of 16384
    int found = 0;
    for (int chunk = 0; chunk < p.n_pages && found < total; chunk += 16384) {
        const int at = chunk + warp * 512 + lane;
        if (chunk > 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                held[i] = at + 32 * i < p.n_pages ? p.refs[at + 32 * i] : 1;
        }
        uint32_t bits[16];
        int mine = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            bits[i] = __ballot_sync(kFull, held[i] == 0);
            mine += __popc(bits[i]);
        }
        int sum;
        int pos = found + warp_prefix(mine, sh, sum);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int k = pos + __popc(bits[i] & ((1u << lane) - 1u));
            if (((bits[i] >> lane) & 1u) && k < total)
                list[k] = at + 32 * i;
            pos += __popc(bits[i]);
        }
        found += sum;
    }
    __syncthreads();
    // (D)
    for (int t = warp; t < tasks; t += 32) {
        const uint32_t m = marks[t];
        if (m == 0)
            continue;
        const int b = owner(t);
        if (count[task0[b + 1]] > found || !((m >> lane) & 1u))
            continue;
        const int c = first[b] + 32 * (t - task0[b]) + lane;
        int32_t *entry = p.table + static_cast<size_t>(b) * p.max_pages + c;
        const int page = list[count[t] + __popc(m & ((1u << lane) - 1u))], old = *entry;
        *entry = page;
        p.refs[page] = 1;
        if (old >= 0 && old < p.n_pages) {
            atomicSub(p.refs + old, 1);
            if (c == first[b])
                s.copies[b] = make_int4(page, old, tail[b], 0);
        }
    }
    if (tid < p.batch) {
        const int upto = count[task0[tid + 1]];
        // (a page that this sequence keeps because the others leave it: pages run out in order, so
        // that if the last of them is served all are)
        const bool fits = (upto == count[task0[tid]] || upto <= found) &&
                          (lean[tid] < 0 || count[task0[lean[tid] + 1]] <= found);
        if (!fits)
            raise_error(p.err, 0x10u);  // SFI_DEVERR_POOL
        if (ok)
            ok[tid] = state[tid] == 0 && fits ? 1 : 0;
    }
}

// The rows of the pages that reserve_kernel replaced: grid (batch, layers, K or V).
__global__ void __launch_bounds__(256) copy_rows_kernel(const PageParams p, const PageScratch s,
                                                        uint4 *k, uint4 *v)
{
    pdl_wait();
    const int4 c = s.copies[blockIdx.x];
    if (c.z == 0)
        return;
    uint4 *t = blockIdx.z ? v : k;
    const size_t page = static_cast<size_t>(p.n_kv_heads) * 256, layer = blockIdx.y * (page * p.n_pages);
    uint4 *to = t + layer + c.x * page;
    const uint4 *from = t + layer + c.y * page;
    const int n = c.z * 16;   // 16-byte pieces of one head's rows
    for (int i = threadIdx.x; i < n * p.n_kv_heads; i += 256) {
        const int at = (i / n) * 256 + i % n;
        to[at] = from[at];
    }
}

// ------------------------------------------------------------------------------ compaction

// One CTA: U = pages in use, the free ids below U and the used ids from U on, both ascending,
// so that the i-th of one goes to the i-th of the other; rank[id] is that i for a used id.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const PageParams p,
                                                                    int32_t *n_used,
                                                                    const PageScratch s)
{
    __shared__ int sh[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    // occupancy of a chunk of 16384 pages, a warp 512 of them; the first chunk's is kept
    auto occupied = [&](int chunk, uint32_t *bits) {
        const int at = chunk + warp * 512 + lane;
        int held[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            held[i] = at + 32 * i < p.n_pages ? p.refs[at + 32 * i] : 0;
        int mine = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            bits[i] = __ballot_sync(kFull, held[i] != 0);
            mine += __popc(bits[i]);
        }
        return mine;
    };
    uint32_t bits[16];
    int used = 0, sum;
    for (int chunk = (p.n_pages - 1) / 16384 * 16384; chunk >= 0; chunk -= 16384)
        used += occupied(chunk, bits);      // (the first chunk last: its bits stay)
    warp_prefix(used, sh, sum);
    const int U = sum;
    int holes = 0, movers = 0;
    for (int chunk = 0; chunk < p.n_pages; chunk += 16384) {
        if (chunk > 0)
            occupied(chunk, bits);
        const int at0 = chunk + warp * 512;
        int mine = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            // below U the free ids count, from U on the used ones
            const int left = U - (at0 + 32 * i);
            const uint32_t below = left >= 32 ? kFull : left <= 0 ? 0u : (1u << left) - 1u;
            bits[i] = (~bits[i] & below) | (bits[i] & ~below);
            mine += __popc(bits[i] & below) + (__popc(bits[i] & ~below) << 16);
        }
        // both counts of a chunk in one word: at most 16384 each
        const int pos = warp_prefix(mine, sh, sum);
        int h = holes + (pos & 0xffff), m = movers + (pos >> 16);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int left = U - (at0 + 32 * i), id = at0 + 32 * i + lane;
            const uint32_t below = left >= 32 ? kFull : left <= 0 ? 0u : (1u << left) - 1u;
            const uint32_t hb = bits[i] & below, mb = bits[i] & ~below, lower = (1u << lane) - 1u;
            if ((hb >> lane) & 1u)
                s.list[h + __popc(hb & lower)] = id;
            if ((mb >> lane) & 1u) {
                s.movers[m + __popc(mb & lower)] = id;
                s.rank[id] = m + __popc(mb & lower);
            }
            h += __popc(hb);
            m += __popc(mb);
        }
        holes += sum & 0xffff;
        movers += sum >> 16;
    }
    if (tid == 0) {
        *n_used = U;
        s.n_moves[0] = movers;
        s.n_moves[1] = U;
    }
}

// Tables, counts and the moved pages: one 4 KB piece (a head's page) per warp step.
__global__ void __launch_bounds__(256) compact_move_kernel(const PageParams p, const PageScratch s,
                                                           uint4 *k, uint4 *v, int n_layers)
{
    pdl_wait();
    const long long threads = static_cast<long long>(gridDim.x) * 256;
    const long long t0 = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const long long entries = static_cast<long long>(p.batch) * p.max_pages;
    const int moves = s.n_moves[0], U = s.n_moves[1];
    for (long long i = t0; i < moves; i += threads) {
        const int from = s.movers[i], to = s.list[i];
        p.refs[to] = p.refs[from];
        p.refs[from] = 0;
    }
    for (long long i = t0; i < entries; i += threads) {
        const int e = p.table[i];
        if (e >= p.n_pages)
            raise_error(p.err, 0x1u);
        else if (e >= U) {
            // (an entry whose page counts as free has no rank)
            const int r = s.rank[e];
            if (r >= 0 && r < moves && s.movers[r] == e)
                p.table[i] = s.list[r];
            else
                raise_error(p.err, 0x80u);  // SFI_DEVERR_REFS
        }
    }
    const int lane = threadIdx.x & 31;
    const long long pieces = static_cast<long long>(moves) * n_layers * 2 * p.n_kv_heads;
    const size_t layer = static_cast<size_t>(p.n_pages) * p.n_kv_heads * 256;
    for (long long w = t0 >> 5; w < pieces; w += threads >> 5) {
        const int head = static_cast<int>(w % p.n_kv_heads);
        long long r = w / p.n_kv_heads;
        const int which = static_cast<int>(r & 1);
        r >>= 1;
        const int l = static_cast<int>(r % n_layers), i = static_cast<int>(r / n_layers);
        uint4 *t = (which ? v : k) + l * layer;
        const uint4 *from = t + (static_cast<size_t>(s.movers[i]) * p.n_kv_heads + head) * 256;
        uint4 *to = t + (static_cast<size_t>(s.list[i]) * p.n_kv_heads + head) * 256;
        uint4 x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = __ldcs(from + j * 32 + lane);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            __stcs(to + j * 32 + lane, x[j]);
    }
}

// --------------------------------------------------------------------------- chunk appends

constexpr int kChunkRows = 8;   // rows per CTA

// The new rows are requested before their places are known (a chain of four loads), and the
// warps find the places of the CTA's rows, one each, meanwhile.
__global__ void __launch_bounds__(256) append_chunk_kernel(const ChunkParams p,
                                                           const uint4 *__restrict__ k_new,
                                                           const uint4 *__restrict__ v_new,
                                                           uint4 *__restrict__ k,
                                                           uint4 *__restrict__ v)
{
    __shared__ long long dst[kChunkRows];
    pdl_trigger();
    pdl_wait();
    const int r0 = blockIdx.x * kChunkRows, hkv = p.pg.n_kv_heads, layer = blockIdx.y;
    const int rows = min(kChunkRows, p.n_rows - r0);
    const int per = hkv * 16;   // 16-byte pieces of one row of one tensor
    const long long head = p.pg.page_size ? 16 : p.pg.capacity;   // cache rows between heads
    const long long base = static_cast<long long>(layer) *
                           (p.pg.page_size ? static_cast<long long>(p.pg.n_pages) * hkv * 16
                                           : static_cast<long long>(p.pg.batch) * hkv * p.pg.capacity);
    bool known = false;
    for (int i = threadIdx.x; i < 2 * per || !known; i += 256) {
        const bool is_v = i >= per, on = i < 2 * per;
        const int j = is_v ? i - per : i;
        const uint4 *src = (is_v ? v_new : k_new) +
                           (static_cast<size_t>(layer) * p.n_rows + r0) * per + j;
        uint4 x[kChunkRows];
#pragma unroll
        for (int q = 0; q < kChunkRows; ++q)
            if (on && q < rows)
                x[q] = __ldcs(src + static_cast<size_t>(q) * per);
        if (!known) {   // (every thread's first step)
            const long long d = chunk_dst(p, r0 + (threadIdx.x >> 5), threadIdx.x & 31);
            if ((threadIdx.x & 31) == 0)
                dst[threadIdx.x >> 5] = d;
            __syncthreads();
            known = true;
        }
        if (!on)
            continue;
        uint4 *to = (is_v ? v : k) + (base + (j >> 4) * head) * 16 + (j & 15);
#pragma unroll
        for (int q = 0; q < kChunkRows; ++q)
            if (dst[q] >= 0)
                to[dst[q] * 16] = x[q];
    }
}

// The lengths after the rows: a warp per sequence, which first looks over the chunk's pages. (A
// cluster of CTAs per sequence that wrote the rows and then advanced the length in one launch
// took 9.3 us for 32 sequences of 1 to 40 rows in four layers; the two launches take 7. Long chunks
// were not tried.)
__global__ void __launch_bounds__(1024) advance_kernel(const ChunkParams p)
{
    pdl_trigger();
    pdl_wait();
    advance_lengths(p);
}

// -------------------------------------------------------------------------------- reorder

// The sequences that move, in order: dst in mv[i].x, src in mv[i].y; returns their number.
// Every thread of the block calls it (blocks of at least 32 threads).
__device__ __forceinline__ int moved_list(const int32_t *src, int batch, int2 *mv, int *count,
                                          uint32_t *err, bool report)
{
    if (threadIdx.x < 32) {
        int n = 0;
        for (int b0 = 0; b0 < batch; b0 += 32) {
            const int b = b0 + static_cast<int>(threadIdx.x);
            const int from = b < batch ? src[b] : b;
            const bool bad = from < 0 || from >= batch;
            if (bad && b < batch && report)
                raise_error(err, 0x40u);  // SFI_DEVERR_SEQ
            const bool go = b < batch && !bad && from != b;
            const uint32_t m = __ballot_sync(kFull, go);
            if (go)
                mv[n + __popc(m & ((1u << threadIdx.x) - 1u))] = make_int2(b, from);
            n += __popc(m);
        }
        if (threadIdx.x == 0)
            *count = n;
    }
    __syncthreads();
    return *count;
}

// The int32 matrices [layers][batch][cols] of a sequence's state, permuted over the batch, 32
// columns per CTA: page table (with its reference counts), selections, counts, lengths.
__global__ void __launch_bounds__(256) reorder_ints_kernel(const ReorderParams p)
{
    extern __shared__ int held[];
    __shared__ int2 mv[kMaxBatch];
    __shared__ int n_mv;
    pdl_wait();
    const int n = moved_list(p.src, p.batch, mv, &n_mv, p.err, blockIdx.x == 0);
    int part = 0, slice = blockIdx.x;
    while (slice >= p.ints[part].slices)
        slice -= p.ints[part++].slices;
    const ReorderInts &a = p.ints[part];
    const int per_layer = (a.cols + 31) / 32;
    const int layer = slice / per_layer, c0 = (slice - layer * per_layer) * 32;
    int32_t *t = a.data + static_cast<size_t>(layer) * p.batch * a.cols;
    const int lane = threadIdx.x & 31, c = c0 + lane;
    if (c < a.cols)
        for (int i = threadIdx.x >> 5; i < n; i += 8)
            held[i * 32 + lane] = t[static_cast<size_t>(mv[i].y) * a.cols + c];
    __syncthreads();
    if (c >= a.cols)
        return;
    for (int i = threadIdx.x >> 5; i < n; i += 8) {
        int32_t *e = t + static_cast<size_t>(mv[i].x) * a.cols + c;
        const int now = held[i * 32 + lane];
        if (a.refs) {
            const int was = *e;
            if (was != now) {
                if (now >= p.n_pages || was >= p.n_pages)
                    raise_error(p.err, 0x1u);  // SFI_DEVERR_PAGE_RANGE
                if (now >= 0 && now < p.n_pages)
                    atomicAdd(a.refs + now, 1);
                if (was >= 0 && was < p.n_pages)
                    atomicSub(a.refs + was, 1);
            }
        }
        *e = now;
    }
}

// Bulk rows, [layers][batch][heads][rows_per_head] of 256 bytes, permuted over the batch in
// place. A CTA holds the same few rows of one head of every moving sequence: each of its
// threads reads its 16-byte pieces of them into registers, all at once, and writes them after
// a barrier, so that no other CTA and no scratch is involved. A row moves if it is below the
// source's row count. kPieces: pieces per thread, enough for a whole batch that moves. The
// moves are sorted by source and a thread takes consecutive ones, so that a source of several
// copies (a fork) is read once per thread and not once per copy.
template <int kPieces>
__global__ void __launch_bounds__(256) reorder_rows_kernel(const ReorderParams p, uint4 *k, uint4 *v,
                                                           int rows_per_head, const int32_t *rows,
                                                           int rows_by_unit, int cols_log2)
{
    __shared__ int2 listed[kMaxBatch], mv[kMaxBatch];
    __shared__ int have[kMaxBatch];
    __shared__ int n_mv;
    pdl_wait();
    const int n = moved_list(p.src, p.batch, listed, &n_mv, p.err, false);
    const int layer = blockIdx.y / p.n_kv_heads, head = blockIdx.y - layer * p.n_kv_heads;
    if (static_cast<int>(threadIdx.x) < n) {    // (at most one each)
        const int2 me = listed[threadIdx.x];
        const int count = rows_by_unit
                              ? rows[(static_cast<long long>(layer) * p.batch + me.y) * p.n_kv_heads + head]
                              : rows[me.y];
        int at = 0;
        for (int i = 0; i < n; ++i) {
            const int y = listed[i].y;
            at += y < me.y || (y == me.y && i < static_cast<int>(threadIdx.x));
        }
        mv[at] = me;
        have[at] = count;
    }
    __syncthreads();
    const long long stride = static_cast<long long>(p.n_kv_heads) * rows_per_head * 16;
    uint4 *t = (blockIdx.z ? v : k) + static_cast<long long>(layer) * p.batch * stride +
               static_cast<long long>(head) * rows_per_head * 16;
    const uint32_t col = (blockIdx.x << cols_log2) + (threadIdx.x & ((1u << cols_log2) - 1u));
    // (at most kPieces each: the batch times the columns is at most 256 kPieces)
    const int groups = 256 >> cols_log2, per = (n + groups - 1) / groups;
    const int m0 = (threadIdx.x >> cols_log2) * per;
    uint4 x[kPieces];
    uint32_t live = 0, same = 0;
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
        const int i = m0 + q;
        if (q < per && i < n && static_cast<int>(col >> 4) < min(have[i], rows_per_head)) {
            live |= 1u << q;
            if (q > 0 && mv[i - 1].y == mv[i].y)
                same |= 1u << q;
            else
                x[q] = t[mv[i].y * stride + col];
        }
    }
#pragma unroll
    for (int q = 1; q < kPieces; ++q)
        if ((same >> q) & 1u)
            x[q] = x[q - 1];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kPieces; ++q)
        if ((live >> q) & 1u)
            t[mv[m0 + q].x * stride + col] = x[q];
}

}  // namespace

cudaError_t launch_drop_pages(const PageParams &p, int evict, int n_sink, int n_window,
                              cudaStream_t stream)
{
    const cudaError_t e = launch_pdl(drop_pages_kernel, dim3((p.max_pages + 255) / 256, p.batch),
                                     dim3(256), 0, stream, p, evict, n_sink, n_window);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_reserve(const PageParams &p, const int32_t *n_new, uint8_t *ok,
                           const PageScratch &s, void *k, void *v, int n_layers,
                           cudaStream_t stream)
{
    cudaError_t e = launch_pdl(reserve_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p, n_new, ok, s);
    if (e == cudaSuccess)
        e = launch_pdl(copy_rows_kernel, dim3(p.batch, n_layers, 2), dim3(256), 0, stream, p, s,
                       static_cast<uint4 *>(k), static_cast<uint4 *>(v));
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_pages_compact(const PageParams &p, int32_t *n_used, const PageScratch &s, void *k,
                                 void *v, int n_layers, int grid, cudaStream_t stream)
{
    cudaError_t e = launch_pdl(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p, n_used, s);
    if (e == cudaSuccess)
        e = launch_pdl(compact_move_kernel, dim3(grid), dim3(256), 0, stream, p, s,
                       static_cast<uint4 *>(k), static_cast<uint4 *>(v), n_layers);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_append_chunk(const ChunkParams &p, const void *k_new, const void *v_new, void *k,
                                void *v, int n_layers, cudaStream_t stream)
{
    const cudaError_t e = launch_pdl(append_chunk_kernel, dim3((p.n_rows + kChunkRows - 1) / kChunkRows, n_layers),
                   dim3(256), 0, stream, p, static_cast<const uint4 *>(k_new),
                   static_cast<const uint4 *>(v_new), static_cast<uint4 *>(k), static_cast<uint4 *>(v));
    return e != cudaSuccess ? e : launch_advance(p, stream);
}

cudaError_t launch_advance(const ChunkParams &p, cudaStream_t stream)
{
    const cudaError_t e = launch_pdl(advance_kernel, dim3(1), dim3(1024), 0, stream, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_reorder_rows(const ReorderParams &p, void *k, void *v, int n_layers,
                                int rows_per_head, const int32_t *rows, int rows_by_unit, cudaStream_t stream)
{
    // pieces per sequence and CTA: a power of two such that the batch fits the threads' registers
    // (8 each, 16 from batch 129 on); at most 256, at least one row
    int lg = 8;
    while (lg > 4 && (p.batch << lg) > 2048)
        --lg;
    const long long pieces = static_cast<long long>(rows_per_head) * 16;
    const dim3 grid(static_cast<unsigned>((pieces + (1 << lg) - 1) >> lg), n_layers * p.n_kv_heads, 2);
    uint4 *kp = static_cast<uint4 *>(k), *vp = static_cast<uint4 *>(v);
    const cudaError_t e =
        (p.batch << lg) <= 2048
            ? launch_pdl(reorder_rows_kernel<8>, grid, dim3(256), 0, stream, p, kp, vp, rows_per_head,
                         rows, rows_by_unit, lg)
            : launch_pdl(reorder_rows_kernel<16>, grid, dim3(256), 0, stream, p, kp, vp, rows_per_head,
                         rows, rows_by_unit, lg);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_reorder_ints(const ReorderParams &p, cudaStream_t stream)
{
    int slices = 0;
    for (int i = 0; i < kReorderParts; ++i)
        slices += p.ints[i].slices;
    const cudaError_t e = launch_pdl(reorder_ints_kernel, dim3(slices), dim3(256),
                                     static_cast<size_t>(p.batch) * 32 * sizeof(int), stream, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sfi
