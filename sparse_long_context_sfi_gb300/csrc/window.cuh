// window.cuh -- attention of a chunk of rows under sinks and a sliding window, straight from
// the cache (contiguous or paged), on the tcgen05 tensor cores; and of rows that see all of another
// sequence (CROSS). One kernel, for window.cu and cross.cu.
//
// A row at position i of query head h sees keys j <= i with j < n_sink or j > i - n_window:
//     z_ij = q_i . k_j / sqrt(128),  o_i = sum_j exp(z_ij - m_i) v_j / sum_j exp(z_ij - m_i).
//
// An item is 256, 128 or 16 operand rows of one (layer, sequence, kv head): its positions times
// the G query heads that share the head's keys, so one read of a K/V row serves the group. The
// keys that any of its rows sees are a list of 16-position blocks (a cache page each): the sink
// blocks, then the blocks of the joint window; a tile is KT / 16 consecutive entries of the
// list, so few sinks share a tile with the window instead of costing one.
//
// One CTA, roles by warp:
//   0      works the items out for all roles; TMA: the item's queries, then K and V of every
//          tile (16-row boxes)
//   1      MMA: S = Q K^T and O += P V per q tile (M = 128), P read from tensor memory
//   2      zeroes the V rows of a landed tile that no row of the item may see (a zero weight
//          would not cancel a NaN)
//   4-7    softmax and output of q tile 0, one row per thread; 8-11 of q tile 1
// Tensor memory: per q tile NS score buffers of KT columns, each overwritten by its weights,
// and 128 columns of O. The running maximum is only moved (and O rescaled) when it grows by
// more than 2^8, so that most tiles leave O alone (an 8K chunk: 491 us with every growth, 417
// without); weights up to 2^8 are as exact in floating point as weights up to 1.
//
// CROSS: rows that see all keys of their sequence. The producer shares the work out as it goes
// (stream_item, or a queue); 32 x 4 rows of 1000 to 4001 keys 59 us (5.0 TB/s; 95 with one CTA to an item),
// 4 x 2048 rows of 8192 keys 765 to 785 us, 1.40 to 1.44 PFLOP/s (751 in a replayed graph; cuBLAS in a loop 1.72).
// fp32 outputs of these 121 and 2447.
//
// Few rows and a long window: the tiles of an item are split over n_split items, whose
// unnormalised outputs, maxima and sums the last one to finish joins, in split order.
//
// What bounds it (GB300, copy rate 6.78 TB/s, bf16 products 1.90 PFLOP/s measured):
//   256 rows, 8K of 32K rows, window 4096: 414 us, 1.33 PFLOP/s (397 in a replayed graph, as are the
//     other figures of this form here). Per 128 keys a q tile's softmax
//     (~2000 clocks), the hand-over of its weights (~370) and their product with the next scores
//     (~1030) are a chain of ~3400, as tensor memory has one score buffer per q tile beside two O
//     (half of whose columns hold nothing while it holds weights: the next scores do not use them);
//     the other q tile fits between, so the tensor core has 2048 clocks of work in 3400 (without
//     the softmax it would take 328 us). An item's start and end cost ~5600 more. Tried: 64-key
//     tiles with two buffers (512 us: smaller products), two threads per score row (429: they
//     share a scheduler, and the weights are handed over later), an MMA warp per q tile (533:
//     the q tiles fall into step), warps of their own for the output (404).
//   128 rows, 4 x 32K rows, window 64: 446 us, 6.0 TB/s of the 2.7 GB it has to move: 335 us
//     without the stores, no less with the softmax left out, 446 with stores through TMA.
//   16 rows, 32 tokens, window 4096, pages: 92 us, 5.9 TB/s. HBM.
//   fp32 outputs: the chunk 1333 us, the prompts 1133, the tokens 186 to 194: one CTA per SM, three
//     products per tile and O into M every second one; of 16 rows one softmax warp is live.
// Registers that spill are the first thing to look at here: shared memory leaves next to no L1,
// so a spill is a trip to L2 (a form that spilled took twice the time).
#pragma once

#include "sfi_device.cuh"

#include <math_constants.h>

#include <climits>
#include <cstddef>
#include <type_traits>

namespace sfi {
namespace {

__device__ __forceinline__ float ex2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// fp32 outputs: tiles summed by the tensor core before O moves to M. Error (2-norm) and time of a
// token of 32 sequences under a window of 4096: every tile 4.9e-7, 238 us; 2 6.6e-7, 194 us;
// 4 1.1e-6, 189 us; never 1.0e-5.
constexpr int kFlush = 2;

// 32 tensor-memory columns of this thread's lane; the values are there after tmem_landed.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
          "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]),
          "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
          "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(addr)
        : "memory");
}

// Wait for this thread's tensor-memory loads. The loaded values go through the statement, so
// that no use of them can be scheduled before it.
__device__ __forceinline__ void tmem_landed(float *v)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                   "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]),
                   "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]),
                   "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]),
                   "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29])
                 :
                 : "memory");
    asm volatile("" : "+f"(v[30]), "+f"(v[31]) : : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
        "%29, %30, %31};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]),
        "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
        "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]),
        "r"(v[31]), "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(addr)
        : "memory");
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

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ void tmem_st_wait()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], bf16 inputs, fp32 accumulate; one thread issues.
__device__ __forceinline__ void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int x,
                                            int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// Polls until `done()` holds in every lane (a warp call; it may test several barriers, whose
// latencies then overlap); gives up like mbar_wait. For the MMA warp, whose waits are on the
// critical path and which has nothing else to do: a wait that is over costs it ~140 clocks.
template <typename F>
__device__ __forceinline__ bool warp_poll(F done, volatile int *abort)
{
    uint64_t t0 = 0;
    for (uint32_t spins = 1;; ++spins) {
        if (__all_sync(0xffffffffu, done()))
            return true;
        if ((spins & 255u) == 0u) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0)
                t0 = now;
            if (__any_sync(0xffffffffu, *abort != 0 || now - t0 > kWaitTimeoutNs))
                return false;
        }
    }
}

// Every lane waits; the answer is the same in all of them.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort)) != 0;
}

// A value that all lanes have, as one that the compiler knows to be uniform over the warp.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_or_sync(0xffffffffu, v); }

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
    return p != 0;
}

// Bits [lo, hi) of word w of a column mask (columns 32 w .. 32 w + 31).
__device__ __forceinline__ uint32_t span_bits(int lo, int hi, int w)
{
    const int a = min(max(lo - 32 * w, 0), 32), b = min(max(hi - 32 * w, 0), 32);
    if (b <= a)
        return 0u;
    return (b == 32 ? 0xffffffffu : ((1u << b) - 1u)) & ~((1u << a) - 1u);
}

constexpr int kMaxStages = 4;

// An item as the producer works it out and the other roles read it.
struct WItem {
    int b, layer, kvh;
    int r0, np, p0;             // first packed row, positions, first position
    int lo;                     // first position of the joint window
    int sb, nb, base;           // sink blocks, all blocks; position = list column + base behind the sinks
    int t0, t1;                 // tiles of this split
    int slot, sp;
    uint32_t row0;              // row of out that the first position and head is
};
// Of rows that see all keys: the sequence's length; the item's first piece, and how many CTAs have
// one. (Fields that an item of the other kind does not have: with them, two q tiles spill.)
struct CPart {
    int end, first, pieces;
};
struct CItem : WItem, CPart {
};
__device__ __forceinline__ int end_of(const WItem &it) { return it.p0 + it.np; }
__device__ __forceinline__ int end_of(const CItem &it) { return it.end; }
__device__ __forceinline__ int first_of(const WItem &) { return 0; }
__device__ __forceinline__ int first_of(const CItem &it) { return it.first; }
__device__ __forceinline__ int pieces_of(const WItem &) { return 1; }
__device__ __forceinline__ int pieces_of(const CItem &it) { return it.pieces; }
constexpr int kItemRing = 4;

struct WCtrl {
    uint64_t kf[kMaxStages], ke[kMaxStages], vf[kMaxStages], vr[kMaxStages], ve[kMaxStages];
    uint64_t qf, qe;
    uint64_t sf[2][2];          // [q tile][score buffer]: scores complete
    uint64_t pf[2][2];          // [q tile][score buffer, or half of the tile's columns with one buffer]:
                                // weights stored (one arrival per softmax warp)
    // an O += P V complete; one per score buffer, because with two the softmax may be two
    // tiles ahead of the products, and one barrier's parity tells only one phase
    uint64_t od[2][2];
    uint64_t oe[2];             // O read out (one arrival per softmax warp)
    uint64_t itf[kItemRing];    // items[i] written
    uint64_t ite[kItemRing];    // and read (one arrival per reading warp)
    uint64_t drain;
    uint64_t gs;                // all softmax warps (splits only)
    uint32_t tmem;
    int abort;
    int last;
    int total;                  // items
    int tiles;                  // q tiles (of 128 NQ rows) of one layer and kv head
    int pre[kMaxBatch + 1];     // q tiles before each sequence (a stream: key tiles of all q tiles)
    int len[kMaxBatch], cnt[kMaxBatch], start[kMaxBatch];
    WItem items[kItemRing];
    CPart parts[kItemRing];
    uint8_t order[kMaxBatch];   // a queue: the sequences, longest first (pre is in this order)
};
constexpr int kWBars = static_cast<int>((offsetof(WCtrl, tmem)) / sizeof(uint64_t));

template <bool CROSS>
using Item = std::conditional_t<CROSS, CItem, WItem>;

template <int ROWS, int KT, bool SPLIT, bool CROSS>
__device__ __forceinline__ Item<CROSS> item_of(const WCtrl &c, const WindowParams &p, int idx)
{
    Item<CROSS> it;
    const int per = ROWS >> p.group_log2;
    // (an integer division costs ~40 instructions: taken only where it says something)
    int q = SPLIT ? idx / p.n_split : idx;
    it.sp = SPLIT ? idx - q * p.n_split : 0;
    const int qh = p.heads_log2 >= 0 ? q >> p.heads_log2 : q / p.n_kv_heads;
    it.kvh = q - qh * p.n_kv_heads;
    q = qh;
    it.layer = p.n_layers == 1 ? 0 : q / c.tiles;
    // the last rows of a prompt first: they see the most keys
    const int t = CROSS ? q - it.layer * c.tiles : c.tiles - 1 - (q - it.layer * c.tiles);
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (c.pre[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int first = (t - c.pre[lo]) * per;
    if (CROSS)
        lo = c.order[lo];
    it.b = lo;
    it.np = min(per, c.cnt[lo] - first);
    it.r0 = c.start[lo] + first;
    if constexpr (CROSS) {      // (a sequence may be empty: no tiles)
        it.p0 = it.lo = it.sb = it.base = 0;
        it.end = c.len[lo];
        it.nb = (it.end + 15) >> 4;
        it.pieces = 1;
    } else {
        it.p0 = c.len[lo] - c.cnt[lo] + first;
        it.lo = max(0, it.p0 - p.n_window + 1);
        const int lo_blk = it.lo >> 4;
        it.sb = min((p.n_sink >> 4) + ((p.n_sink & 15) != 0), lo_blk);
        it.base = (lo_blk - it.sb) * 16;
        it.nb = it.sb + ((it.p0 + it.np - 1) >> 4) - lo_blk + 1;
    }
    const int n = (it.nb + KT / 16 - 1) / (KT / 16);
    it.t0 = 0;
    it.t1 = n;
    if (SPLIT) {                // (tiles * splits stays far below 2^32: at most 2^27 positions of 64)
        it.t0 = static_cast<int>(static_cast<uint32_t>(n) * it.sp / p.n_split);
        it.t1 = static_cast<int>(static_cast<uint32_t>(n) * (it.sp + 1) / p.n_split);
    }
    it.slot = (it.layer * c.tiles + t) * p.n_kv_heads + it.kvh;
    it.row0 = (static_cast<uint32_t>(it.layer * p.n_rows + it.r0) * p.n_kv_heads + it.kvh) << p.group_log2;
    return it;
}

// A stream: the key tiles of all items in a row, unit by unit, sequence by sequence, q tile by q
// tile, with kOver tiles' time in front of each item for its start and end; every CTA has an equal
// share, and an item whose tiles lie in the shares of several is joined.
constexpr int kOver = 2;

struct Stream {
    uint64_t per_unit, total, ctas;
    __device__ __forceinline__ uint64_t start(uint64_t cta) const { return total * cta / ctas; }
    // the CTA whose share has tile g
    __device__ __forceinline__ int owner(uint64_t g) const { return static_cast<int>(((g + 1) * ctas - 1) / total); }
};

// What CTA `cta`, whose share ends at `end`, has of the item at tile g, and where it goes on; np 0: nothing.
template <int ROWS, int KT>
__device__ __forceinline__ CItem stream_item(const WCtrl &c, const WindowParams &p, const Stream &s, uint64_t g,
                                             uint64_t end, int cta, uint64_t &next)
{
    CItem it;
    const int per = ROWS >> p.group_log2;
    const uint64_t unit = g / s.per_unit;
    const uint32_t rem = static_cast<uint32_t>(g - unit * s.per_unit);
    it.layer = static_cast<int>(unit / p.n_kv_heads);
    it.kvh = static_cast<int>(unit) - it.layer * p.n_kv_heads;
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<uint32_t>(c.pre[mid]) <= rem)
            lo = mid;
        else
            hi = mid;
    }
    it.b = lo;
    const uint32_t n = static_cast<uint32_t>(c.len[lo] + KT - 1) / KT, n1 = n + kOver;
    const uint32_t in = rem - static_cast<uint32_t>(c.pre[lo]), tile = in / n1;
    const int first = static_cast<int>(tile) * per, from = static_cast<int>(in - tile * n1);
    it.r0 = c.start[lo] + first;
    it.p0 = it.lo = it.sb = it.base = it.slot = 0;
    it.end = c.len[lo];
    it.nb = (it.end + 15) >> 4;
    const uint64_t begin = g - from, stop = begin + n1;
    next = stop < end ? stop : end;
    it.t0 = max(from - kOver, 0);
    it.t1 = max(static_cast<int>(next - begin) - kOver, 0);
    // (an item without keys is its start's)
    it.np = it.t1 > it.t0 || (n == 0 && from == 0) ? min(per, c.cnt[lo] - first) : 0;
    const int c0 = n > 0 && begin + kOver < s.start(cta) ? s.owner(begin + kOver) : cta;
    const int c1 = n > 0 && stop > end ? s.owner(stop - 1) : cta;
    // pieces: a CTA's first is of the item at its share's start, its second of one that goes on
    it.first = 2 * c0 + (s.start(c0) < begin ? 1 : 0);
    it.sp = c0 == cta ? it.first : 2 * cta;
    it.pieces = c1 - c0 + 1;
    it.row0 = (static_cast<uint32_t>(it.layer * p.n_rows + it.r0) * p.n_kv_heads + it.kvh) << p.group_log2;
    return it;
}

__device__ __forceinline__ void wfail(WCtrl &c, uint32_t *err)
{
    c.abort = 1;
    raise_error(err, 0x4u);  // SFI_DEVERR_TIMEOUT
}

__device__ __forceinline__ void st_global32(void *p, const uint32_t *w)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// N output values of one row, a thread per row: in 32-byte pieces, whole sectors,
// where the output is aligned to them.
template <int N, bool FP32>
__device__ __forceinline__ void store_row(const WindowParams &p, size_t at, const float *v)
{
    if constexpr (FP32) {
        float *o = static_cast<float *>(p.out) + at;
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            const uint32_t *w = reinterpret_cast<const uint32_t *>(v + i);
            if (p.out_aligned32) {
                st_global32(o + i, w);
            } else {
                *reinterpret_cast<uint4 *>(o + i) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4 *>(o + i + 4) = make_uint4(w[4], w[5], w[6], w[7]);
            }
        }
    } else {
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + at;
#pragma unroll
        for (int i = 0; i < N; i += 16) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[i + 2 * j], v[i + 2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t *>(&h);
            }
            if (p.out_aligned32) {
                st_global32(o + i, w);
            } else {
                *reinterpret_cast<uint4 *>(o + i) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4 *>(o + i + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            }
        }
    }
}

// 8 output values, 16-byte aligned.
template <bool FP32>
__device__ __forceinline__ void store_8(const WindowParams &p, size_t at, const float *v)
{
    if constexpr (FP32) {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            h[j] = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + at) = *reinterpret_cast<const uint4 *>(h);
    }
}

// 128 bytes of each of a warp's 32 rows, a thread per row, in four pieces of 32 bytes: the pieces
// are transposed among each four lanes, so that a store instruction covers whole lines of 8 rows
// instead of a sector of each of 32. `at` says where (in bytes) the piece of a row belongs, or
// a negative number for rows that are not written. For the form whose time is its output: four
// 32K prompts under a window of 64 take 450 us, with store_row 472 (and 335 with no store at
// all). With two q tiles the transposition costs the tile loop more than it gives (an 8K chunk
// under a window of 4096: 414 us against 395), with one token it is only latency.
template <typename At>
__device__ __forceinline__ void store_lines(const WindowParams &p, uint32_t *w, int lane, At at)
{
#pragma unroll
    for (int step = 1; step <= 2; ++step) {
        const bool upper = (lane & step) != 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            // pieces (0, 1) and (2, 3), then (0, 2) and (1, 3)
            const int lo = step == 1 ? (i >> 3) * 16 + (i & 7) : i, hi = lo + 8 * step;
            const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? w[lo] : w[hi], step);
            w[lo] = upper ? got : w[lo];
            w[hi] = upper ? w[hi] : got;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long to = at(i);
        if (to < 0)
            continue;
        uint8_t *o = static_cast<uint8_t *>(p.out) + to + 32 * (lane & 3);
        const uint32_t *v = w + 8 * i;
        if (p.out_aligned32) {
            st_global32(o, v);
        } else {
            reinterpret_cast<uint4 *>(o)[0] = make_uint4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<uint4 *>(o)[1] = make_uint4(v[4], v[5], v[6], v[7]);
        }
    }
}

template <int NQ, int KT, int ST, int QR>
constexpr int window_smem() { return 1024 + NQ * QR * 256 + ST * KT * 512 + static_cast<int>(sizeof(WCtrl)); }

// NQ q tiles of QR operand rows, KT keys per tile, ST stages of keys and values, NS score
// buffers per q tile. QR 16 is for single tokens: the MMA still takes 128 rows, of which all
// but the first 16 are whatever lies behind them in shared memory; they end in rows of S and O
// that nobody reads, and the memory holds a third stage instead.
// PARTS: the bf16 parts in which a weight enters the product with V. Single tokens have two, 16
// bits, as in the decode kernels (one token of 32 sequences under a window of 4096: 92 us, with one
// part 87): an output near zero is then off by its own rounding alone. In a chunk's bf16 outputs
// the second part costs more than it gives: four 32K prompts under a window of 64 take 518 us with
// it and 446 without, an 8K chunk under 4096 617 and 412, 4 x 2048 rows that see 8192 states each 1132 and
// 765, ragged ones 113 and 91, and the error (2-norm) falls from 2.2e-3 to 2.3e-3 to the output's own
// rounding, 1.7e-3; fp32 outputs are there for who needs more.
// F32 (fp32 outputs): three parts, 24 bits, and O is moved every kFlush tiles to a second
// accumulator M with ordinary additions: the tensor core's own additions do not round to nearest,
// and 520 of them in a row (two parts, a window of 4096) had left outputs 1.0e-5 off (2-norm). Tensor
// memory then holds one CTA per SM. A bf16 output rounds at 2^-8 and does not need M.
// SPLIT: an item's keys over several CTAs (the joining code costs registers).
template <int NQ, int KT, int ST, int NS, int QR, int PARTS, bool F32, bool SPLIT, bool CROSS>
__global__ void __launch_bounds__(128 + 128 * NQ, NQ == 1 && !F32 ? 2 : 1)
    window_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ CUtensorMap tm_q, const WindowParams p)
{
    constexpr int kRows = NQ * QR, kHalfQ = QR * 128, kHalfKV = KT * 128, kStage = 4 * kHalfKV, kBlocks = KT / 16;
    constexpr uint32_t kCols = NQ == 1 && !F32 ? 256 : 512;
    constexpr int kSW = F32 ? KT + KT / 2 : KT;     // columns of a score buffer
    constexpr int kQTile = NS * kSW + (F32 ? 256 : 128);     // and of a q tile with O (and M)
    constexpr int NH = NS == 1 ? 2 : 1;     // parts in which a tile's weights are handed over
    // Rows that see all keys are shared out by the producer, as it goes: in equal shares of all key
    // tiles, or as a queue of whole items, longest first. The other roles take items until one is empty.
    constexpr bool kStream = SPLIT && CROSS, kFed = CROSS;
    static_assert(NQ * kQTile <= static_cast<int>(kCols) && ST <= kMaxStages && NS <= 2);
    static_assert(!F32 || NQ == 1);
    static_assert((PARTS == 3) == F32 && PARTS >= 1 && PARTS <= 3);
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint8_t *kv_smem = smem + NQ * 2 * kHalfQ;
    WCtrl &c = *reinterpret_cast<WCtrl *>(kv_smem + ST * kStage);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.group, per = kRows >> p.group_log2;

    if (tid < kWBars) {
        uint64_t *bar = reinterpret_cast<uint64_t *>(&c) + tid;
        const int off = tid * 8;
        const bool four = (off >= static_cast<int>(offsetof(WCtrl, pf)) && off < static_cast<int>(offsetof(WCtrl, od))) ||
                          (off >= static_cast<int>(offsetof(WCtrl, oe)) && off < static_cast<int>(offsetof(WCtrl, itf)));
        const bool readers = off >= static_cast<int>(offsetof(WCtrl, ite)) && off < static_cast<int>(offsetof(WCtrl, drain));
        mbar_init(bar, off == static_cast<int>(offsetof(WCtrl, gs)) ? 4 * NQ : readers ? 4 * NQ + 2 : four ? 4 : 1);
        mbar_fence_init();
    }
    if (warp == 1) {
        tmem_alloc(&c.tmem, kCols);
        tmem_relinquish();
    }
    if (tid == 0) {
        c.abort = 0;
        tma_prefetch_map(&tm_k);
        tma_prefetch_map(&tm_v);
        tma_prefetch_map(&tm_q);
    }
    pdl_trigger();
    pdl_wait();
    // the chunk: every sequence's rows and q tiles
    for (int b = tid; b < p.batch; b += 128 + 128 * NQ) {
        const int s0 = p.row_start ? p.row_start[b] : b, s1 = p.row_start ? p.row_start[b + 1] : b + 1;
        const int L = p.seq_len[b];
        int n = s1 - s0;
        if (p.active && !p.active[b]) {
            n = 0;
        } else {
            if (s0 < 0 || n < 0 || s1 > p.n_rows || n > p.max_rows) {
                n = 0;
                if (blockIdx.x == 0)
                    raise_error(p.err, 0x20u);  // SFI_DEVERR_ROWS
            } else if (L < (CROSS ? 0 : n) || L > p.max_len) {
                n = -1 - n;     // (told below, if its rows are its own)
            }
        }
        c.cnt[b] = n;
        c.len[b] = L;
        c.start[b] = s0;
    }
    __syncthreads();
    if (warp == 0) {
        // Where row_start runs backwards somewhere, rows belong to the first sequence that claims
        // them: one that begins before an earlier start is skipped (so that there are never more
        // items than the rows can hold).
        int run = 0, high = INT_MIN;
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
            const int b = b0 + lane;
            const int s0 = b < p.batch ? c.start[b] : INT_MIN;
            int upto = s0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1)
                upto = max(upto, __shfl_up_sync(0xffffffffu, upto, o));
            int n = b < p.batch ? c.cnt[b] : 0;
            const uint32_t bad = n != 0 && n != -1 && max(high, upto) > s0 ? 0x20u  // SFI_DEVERR_ROWS
                                 : n < 0                                   ? 0x8u   // SFI_DEVERR_LENGTH
                                                                           : 0u;
            if (bad) {
                c.cnt[b] = n = 0;
                if (blockIdx.x == 0)
                    raise_error(p.err, bad);
            }
            high = max(high, __shfl_sync(0xffffffffu, upto, 31));
            int v = (n + per - 1) / per;
            if (kStream)
                v *= (b < p.batch ? (c.len[b] + KT - 1) / KT : 0) + kOver;
            int x = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o)
                    x += y;
            }
            if (b < p.batch)
                c.pre[b] = run + x - v;
            run += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) {
            c.tiles = run;
            c.total = kStream ? run : run * p.n_kv_heads * p.n_layers * p.n_split;
        }
    }
    if constexpr (CROSS && !SPLIT) {
        // the queue's order: longest first, and the q tiles in front of each
        __syncthreads();
        for (int b = tid; b < p.batch; b += 128 + 128 * NQ) {
            const int mine = c.len[b];
            int at = 0;
            for (int o = 0; o < p.batch; ++o)
                at += c.len[o] > mine || (c.len[o] == mine && o < b);
            c.order[at] = static_cast<uint8_t>(b);
        }
        __syncthreads();
        if (warp == 0) {
            int run = 0;
            for (int b0 = 0; b0 < p.batch; b0 += 32) {
                const int b = b0 + lane, v = b < p.batch ? (c.cnt[c.order[b]] + per - 1) / per : 0;
                int x = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o)
                        x += y;
                }
                if (b < p.batch)
                    c.pre[b] = run + x - v;
                run += __shfl_sync(0xffffffffu, x, 31);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c.tmem;
    const int total = c.total;
    auto s_col = [&](int a, int buf) { return tmem + a * kQTile + buf * kSW; };
    auto o_col = [&](int a) { return tmem + a * kQTile + NS * kSW; };

    // The n-th item of this CTA, for the roles other than the producer: what they do not use of it
    // is never read. False if the wait ran out.
    auto next_item = [&](uint32_t n, Item<CROSS> &it) -> bool {
        if (!warp_wait(&c.itf[n % kItemRing], (n / kItemRing) & 1, &c.abort))
            return false;
        static_cast<WItem &>(it) = c.items[n % kItemRing];
        if constexpr (CROSS)
            static_cast<CPart &>(it) = c.parts[n % kItemRing];
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&c.ite[n % kItemRing]);
        return true;
    };
    uint32_t syncs = 0;
    constexpr int kOut0 = 128;      // the first softmax thread
    auto out_sync = [&]() -> bool {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&c.gs);
        return warp_wait(&c.gs, syncs++ & 1, &c.abort);
    };
    // O of q tile a once its `done`-th tile's product is complete, divided and written (or left as
    // a partial and joined); each thread a row. False if a wait ran out.
    auto finish = [&](int a, const Item<CROSS> &it, uint32_t done, float m, float l) -> bool {
        const int quad = warp & 3, rq = a * 128 + quad * 32 + lane;
        const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
        const int dp = rq >> p.group_log2, h = rq & (G - 1), nrows = it.np * G;
        const bool valid = rq < nrows, live = a * 128 + quad * 32 < nrows;
        const size_t part = kStream ? it.sp : SPLIT ? static_cast<size_t>(it.slot) * p.n_split + it.sp : 0;
        const bool cut = kStream ? pieces_of(it) > 1 : SPLIT;
        if (it.t1 > it.t0) {
            const size_t my_row = it.row0 + dp * (p.n_kv_heads * G) + h;
            const float inv = cut ? 1.f : 1.f / l;
            if (!warp_wait(&c.od[a][(done - 1) % NS], ((done - 1) / NS) & 1, &c.abort))
                return false;
            tc_fence_after();
            auto release = [&] {        // O is free for the next item
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&c.oe[a]);
            };
            if (live) {
                // (the arrays inside the branch: defined on one path only, they would count as live
                // around the whole loop over items)
                float o[2][32];         // 32 columns at a time, the next ones on their way
                constexpr bool kLines = NQ == 1 && QR == 128 && !F32;
                uint32_t line[kLines ? 32 : 1];     // 128 bytes of the row
                tmem_ld32(o_col(a) + lane_addr, o[0]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float *v = o[q & 1];
                    tmem_landed(v);
                    if constexpr (F32) {
                        if (it.t1 - it.t0 > kFlush) {
                            float mm[32];
                            tmem_ld32(o_col(a) + 128 + lane_addr + 32 * q, mm);
                            tmem_landed(mm);
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                v[x] += mm[x];
                        }
                    }
                    if (q < 3)
                        tmem_ld32(o_col(a) + lane_addr + 32 * q + 32, o[(q + 1) & 1]);
                    else
                        release();
                    if (kLines && !cut) {
                      if constexpr (kLines) {
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * x] * inv, v[2 * x + 1] * inv);
                            line[16 * (q & 1) + x] = *reinterpret_cast<const uint32_t *>(&b);
                        }
                        if (q & 1)
                            store_lines(p, line, lane, [&](int i) -> long long {
                                const int r = (rq & ~3) + i;
                                const uint32_t row = it.row0 + (r >> p.group_log2) * (p.n_kv_heads * G) + (r & (G - 1));
                                return r < nrows ? static_cast<long long>(row) * 256 + 64 * (q - 1) : -1;
                            });
                      }
                    } else if (valid && !cut) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            v[x] *= inv;
                        store_row<32, F32>(p, my_row * kHeadDim + 32 * q, v);
                    } else if (valid) {
                        float *w = p.parts + (part * p.part_rows + rq) * kHeadDim + 32 * q;
#pragma unroll
                        for (int x = 0; x < 32; x += 8)
                            st_global32(w + x, reinterpret_cast<const uint32_t *>(v + x));
                    }
                }
            } else {
                release();
            }
        } else if (CROSS && !cut && valid) {        // nothing to see
            const float none[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            const size_t my_row = it.row0 + dp * (p.n_kv_heads * G) + h;
#pragma unroll 1
            for (int d = 0; d < kHeadDim; d += 8)
                store_8<F32>(p, my_row * kHeadDim + d, none);
        }
        if (SPLIT && cut) {
            if (valid)
                p.part_ml[part * p.part_rows + rq] = make_float2(m, l);
            // every thread's partials before the ticket, the ticket before any read
            __threadfence();
            if (!out_sync())
                return false;
            const int pieces = kStream ? pieces_of(it) : p.n_split;
            int *ticket = p.tickets + (kStream ? first_of(it) >> 1 : it.slot);
            if (tid == kOut0)
                c.last = atomic_add_acq_rel_gpu(ticket, 1) == pieces - 1;
            if (!out_sync())
                return false;
            if (c.last != 0) {
                if (tid == kOut0)
                    *ticket = 0;
                __threadfence();
                if constexpr (kStream) {
                    // 32 threads a row, 4 dims each; several rows' loads on their way at once, pieces in
                    // order of their CTAs, relative to the running maximum
                    constexpr int kRowsAtOnce = 4;
                    const int d = (tid - kOut0) & 31, w0 = (tid - kOut0) >> 5;
                    for (int r0 = w0; r0 < nrows; r0 += 4 * NQ * kRowsAtOnce) {
                        float4 acc[kRowsAtOnce];
                        float top[kRowsAtOnce], den[kRowsAtOnce];
#pragma unroll
                        for (int i = 0; i < kRowsAtOnce; ++i) {
                            acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                            top[i] = -CUDART_INF_F;
                            den[i] = 0.f;
                        }
#pragma unroll 2
                        for (int sp = 0; sp < pieces; ++sp) {
                            const size_t at = (sp == 0 ? static_cast<size_t>(first_of(it))
                                                       : static_cast<size_t>(first_of(it) & ~1) + 2 * sp) * p.part_rows;
                            float2 ml[kRowsAtOnce];
                            float4 v[kRowsAtOnce];
#pragma unroll
                            for (int i = 0; i < kRowsAtOnce; ++i) {
                                const size_t r = at + min(r0 + 4 * NQ * i, nrows - 1);
                                ml[i] = __ldcg(p.part_ml + r);
                                v[i] = __ldcg(reinterpret_cast<const float4 *>(p.parts + r * kHeadDim) + d);
                            }
#pragma unroll
                            for (int i = 0; i < kRowsAtOnce; ++i) {
                                const float mn = fmaxf(top[i], ml[i].x);
                                // (a piece whose maximum is not there counts as it is: its sum is not a number)
                                const float was = mn == -CUDART_INF_F ? 1.f : ex2_approx((top[i] - mn) * p.scale_log2);
                                const float is = mn == -CUDART_INF_F ? 1.f : ex2_approx((ml[i].x - mn) * p.scale_log2);
                                acc[i].x = fmaf(is, v[i].x, acc[i].x * was);
                                acc[i].y = fmaf(is, v[i].y, acc[i].y * was);
                                acc[i].z = fmaf(is, v[i].z, acc[i].z * was);
                                acc[i].w = fmaf(is, v[i].w, acc[i].w * was);
                                den[i] = fmaf(is, ml[i].y, den[i] * was);
                                top[i] = mn;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < kRowsAtOnce; ++i) {
                            const int r = r0 + 4 * NQ * i;
                            if (r >= nrows)
                                continue;
                            const size_t o = static_cast<size_t>(it.row0 + (r >> p.group_log2) * (p.n_kv_heads * G) +
                                                                 (r & (G - 1))) * kHeadDim + 4 * d;
                            const float inv = 1.f / den[i];
                            if constexpr (F32) {
                                *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + o) =
                                    make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv);
                            } else {
                                const __nv_bfloat162 h[2] = {__floats2bfloat162_rn(acc[i].x * inv, acc[i].y * inv),
                                                             __floats2bfloat162_rn(acc[i].z * inv, acc[i].w * inv)};
                                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + o) =
                                    *reinterpret_cast<const uint2 *>(h);
                            }
                        }
                    }
                    return true;
                }
                // a thread per (row, dim): 128 dims, NQ rows at a time; splits in order
                const int d = (tid - kOut0) & 127;
                for (int r = (tid - kOut0) >> 7; r < nrows; r += NQ) {
                    const size_t p0 = static_cast<size_t>(it.slot) * p.n_split * p.part_rows + r;
                    float M = -CUDART_INF_F;
                    for (int sp = 0; sp < p.n_split; ++sp)
                        M = fmaxf(M, __ldcg(p.part_ml + p0 + static_cast<size_t>(sp) * p.part_rows).x);
                    float acc = 0.f, den = 0.f;
                    for (int sp = 0; sp < p.n_split; ++sp) {
                        const size_t at = p0 + static_cast<size_t>(sp) * p.part_rows;
                        const float2 ml = __ldcg(p.part_ml + at);
                        // (a split that saw nothing left no outputs; one whose sum is not a number did)
                        if (ml.y != 0.f) {
                            const float w = ex2_approx((ml.x - M) * p.scale_log2);
                            acc = fmaf(w, __ldcg(p.parts + at * kHeadDim + d), acc);
                            den = fmaf(w, ml.y, den);
                        }
                    }
                    const int dpr = r >> p.group_log2;
                    const size_t o = static_cast<size_t>(it.row0 + dpr * (p.n_kv_heads * G) + (r & (G - 1))) *
                                         kHeadDim + d;
                    if (F32)
                        static_cast<float *>(p.out)[o] = acc / den;
                    else
                        static_cast<__nv_bfloat16 *>(p.out)[o] = __float2bfloat16_rn(acc / den);
                }
            }
        }
        return true;
    };

    // Registers (launched with 168 a thread, or 128 with two CTAs per SM): the softmax keeps a
    // score row, the other roles give up what they do not need. 384 * 168 = 256 * 184 + 128 * 136;
    // 256 * 128 = 128 * 192 + 128 * 64. (With F32 everybody has enough.)
    if (warp >= 4) {
        if constexpr (!F32)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(NQ == 1 ? 192 : 184));
        // ------------------------------------------------------------------------ softmax
        const int a = (warp - 4) >> 2, quad = warp & 3, rowi = quad * 32 + lane;
        const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
        const float sc = p.scale_log2;
        uint32_t done = 0;              // tiles so far, all items
        bool ok = true;
        const int rq = a * 128 + rowi;
        uint32_t nth = 0;
        for (int idx = blockIdx.x; kFed || idx < total; idx += gridDim.x, ++nth) {
            Item<CROSS> it;
            ok = next_item(nth, it);
            if (!ok || (kFed && it.np == 0))
                break;
            const int dp = rq >> p.group_log2;
            const bool valid = dp < it.np;
            const bool live = a * 128 + quad * 32 < it.np * G;   // some row of the warp is valid
            const int i = it.p0 + dp;                       // this row's position
            // it sees the list columns [0, e1) and [a2, e2)
            const int e1 = CROSS ? 0 : min(p.n_sink, i + 1);
            const int a2 = CROSS ? 0 : max(i - p.n_window + 1, 0) - it.base, e2 = CROSS ? end_of(it) : i - it.base + 1;
            float m = -CUDART_INF_F, l = 0.f;
            for (int t = it.t0; t < it.t1; ++t, ++done) {
                const int buf = done % NS;
                ok = warp_wait(&c.sf[a][buf], (done / NS) & 1, &c.abort);
                if (!ok)
                    break;
                tc_fence_after();
                if (!live) {
                    // (the product takes what lies there, into rows that nobody reads)
                    if (lane == 0) {
                        if (NH == 2)
                            mbar_arrive(&c.pf[a][0]);
                        mbar_arrive(&c.pf[a][NH == 2 ? 1 : buf]);
                    }
                    continue;
                }
                const uint32_t sa = s_col(a, buf) + lane_addr;
                const int c0 = t * KT;
                const bool whole = __all_sync(0xffffffffu, a2 <= c0 && e2 >= c0 + KT);
                // 64 columns of scores stay in registers from the maximum to the weights; of a
                // 128-column tile the other 64 are looked at first and read again later, which
                // costs less than the registers of a whole row (spills go to L2 here: shared
                // memory leaves next to no L1).
                constexpr int kC = KT / 32;
                float s[64];
                uint32_t hidden = 0;        // 32-column chunks that no row of the warp sees
                // chunk q, its columns that the row does not see at -inf
                auto mask = [&](float *v, int q) {
                    const uint32_t see = span_bits(0, e1 - c0, q) | span_bits(a2 - c0, e2 - c0, q);
                    if (!__any_sync(0xffffffffu, valid && see != 0u)) {
                        hidden |= 1u << q;
                    } else if (!__all_sync(0xffffffffu, see == 0xffffffffu)) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            v[x] = (see >> x) & 1u ? v[x] : -CUDART_INF_F;
                    }
                };
                float mx[4] = {m, m, m, m};
#pragma unroll
                for (int q0 = kC - 2; q0 >= 0; q0 -= 2) {
                    tmem_ld32(sa + 32 * q0, s);
                    tmem_ld32(sa + 32 * q0 + 32, s + 32);
                    tmem_landed(s);
                    tmem_landed(s + 32);
                    if (!whole) {
                        mask(s, q0);
                        mask(s + 32, q0 + 1);
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        if ((hidden >> (q0 + q)) & 1u)
                            continue;
#pragma unroll
                        for (int x = 0; x < 32; x += 8) {
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                mx[y] = max3(mx[y], s[32 * q + x + 2 * y], s[32 * q + x + 2 * y + 1]);
                        }
                    }
                }
                const float mn = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                const bool grow = (mn - m) * sc > 8.f;      // (from -inf: always, unless still -inf)
                const int nth_tile = t - it.t0;
                const bool flush = F32 && nth_tile > 0 && nth_tile % kFlush == 0;
                if (flush || (__any_sync(0xffffffffu, grow) && nth_tile > 0)) {
                    // O (and M) to the new maximum, O into M
                    const float alpha = grow ? ex2_approx((m - mn) * sc) : 1.f;
                    ok = warp_wait(&c.od[a][(done - 1) % NS], ((done - 1) / NS) & 1, &c.abort);
                    if (!ok)
                        break;
                    tc_fence_after();
                    l *= alpha;
                    const bool has_m = F32 && nth_tile > kFlush;    // M holds something
#pragma unroll(F32 ? 1 : 4)
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t oa = o_col(a) + lane_addr + 32 * q;
                        float o[32], mm[F32 ? 32 : 1];
                        tmem_ld32(oa, o);
                        if constexpr (F32) {
                            if (has_m)
                                tmem_ld32(oa + 128, mm);
                            else
#pragma unroll
                                for (int x = 0; x < 32; ++x)
                                    mm[x] = 0.f;
                            tmem_landed(mm);
                        }
                        tmem_landed(o);
                        if (flush) {
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                o[x] = (o[x] + mm[F32 ? x : 0]) * alpha;
                            tmem_st32(oa + 128, reinterpret_cast<const uint32_t *>(o));
                        } else {
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                o[x] *= alpha;
                            tmem_st32(oa, reinterpret_cast<const uint32_t *>(o));
                            if constexpr (F32) {
                                if (has_m) {
#pragma unroll
                                    for (int x = 0; x < 32; ++x)
                                        mm[x] *= alpha;
                                    tmem_st32(oa + 128, reinterpret_cast<const uint32_t *>(mm));
                                }
                            }
                        }
                    }
                }
                m = grow ? mn : m;
                const float off = m == -CUDART_INF_F ? 0.f : -m * sc;
                const uint64_t sc2 = pack2(sc, sc), off2 = pack2(off, off);
                uint64_t sum = 0;
                // Weights of chunk q over the first 16 columns of its scores; their remainders over the
                // other 16, and what those leave behind the scores. (Stores of 16 columns: with 8 the
                // 8K chunk under a window of 4096 took 417 us, with 16 397, with 32 no less.)
#pragma unroll
                for (int q = 0; q < kC; ++q) {
                    float *v = s + 32 * (q & 1);
                    if (q >= 2) {
                        tmem_landed(v);
                        if (!whole)
                            mask(v, q);
                    }
                    uint32_t w[16], r[PARTS > 1 ? 16 : 1], r2[PARTS > 2 ? 16 : 1];
                    if ((hidden >> q) & 1u) {
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            w[x] = r[PARTS > 1 ? x : 0] = r2[PARTS > 2 ? x : 0] = 0u;
                    } else {
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const float2 z = unpack2(fma2(pack2(v[2 * x], v[2 * x + 1]), sc2, off2));
                            const float p0 = ex2_approx(z.x), p1 = ex2_approx(z.y);
                            sum = add2(sum, pack2(p0, p1));
                            const __nv_bfloat162 hi = __floats2bfloat162_rn(p0, p1);
                            w[x] = *reinterpret_cast<const uint32_t *>(&hi);
                            if (PARTS > 1) {
                                // (the differences are exact)
                                const float2 b = __bfloat1622float2(hi);
                                const float d0 = p0 - b.x, d1 = p1 - b.y;
                                const __nv_bfloat162 lo = __floats2bfloat162_rn(d0, d1);
                                r[PARTS > 1 ? x : 0] = *reinterpret_cast<const uint32_t *>(&lo);
                                if (PARTS > 2) {
                                    const float2 e = __bfloat1622float2(lo);
                                    const __nv_bfloat162 rest = __floats2bfloat162_rn(d0 - e.x, d1 - e.y);
                                    r2[PARTS > 2 ? x : 0] = *reinterpret_cast<const uint32_t *>(&rest);
                                }
                            }
                        }
                    }
                    if (NH == 2 && q == kC / 2) {
                        // the first half of the weights has been stored for a while: let its
                        // product go
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&c.pf[a][0]);
                    }
                    tmem_st16(sa + 32 * q, w);
                    if (PARTS > 1)
                        tmem_st16(sa + 32 * q + 16, r);
                    if (PARTS > 2)
                        tmem_st16(sa + KT + 16 * q, r2);
                    if (q + 2 < kC)
                        tmem_ld32(sa + 32 * q + 64, v);
                }
                const float2 sums = unpack2(sum);
                l += sums.x + sums.y;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&c.pf[a][NH == 2 ? 1 : buf]);
            }
            if (!ok)
                break;
            ok = finish(a, it, done, m, l);
            if (!ok)
                break;
        }
        if (!ok && lane == 0)
            wfail(c, p.err);
    } else {
        if constexpr (!F32)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(NQ == 1 ? 64 : 136));
        if (warp == 0) {
            // ------------------------------------------------------------------ TMA producer
            int use = 0, items = 0;
            bool ok = true;
            uint32_t nth = 0;
            Stream stream = {};
            uint64_t g = 0, g_end = 0;
            if constexpr (kStream) {
                // (as many CTAs as have p.n_split tiles each)
                stream.per_unit = static_cast<uint32_t>(total);
                stream.total = stream.per_unit * static_cast<uint32_t>(p.n_kv_heads * p.n_layers);
                const uint64_t most = (stream.total + p.n_split - 1) / p.n_split;
                stream.ctas = most < gridDim.x ? most : gridDim.x;
                if (blockIdx.x < stream.ctas) {
                    g = stream.start(blockIdx.x);
                    g_end = stream.start(blockIdx.x + 1);
                }
            }
            bool over = false;          // the item that says so is out
            int ahead = 0;              // the queue's next item
            for (int idx = blockIdx.x; (kFed ? !over : idx < total) && ok; idx = CROSS && !SPLIT ? ahead : idx + gridDim.x, ++nth) {
                Item<CROSS> it;
                if constexpr (kStream) {
                    do {
                        over = g >= g_end;
                        if (over)
                            it.np = 0;
                        else
                            it = stream_item<kRows, KT>(c, p, stream, g, g_end, blockIdx.x, g);
                    } while (!over && it.np == 0);
                } else if constexpr (CROSS) {
                    over = idx >= total;
                    if (over) {
                        it.np = 0;
                    } else {
                        if (lane == 0)
                            ahead = static_cast<int>(gridDim.x) + atomicAdd(p.tickets, 1);
                        ahead = __shfl_sync(0xffffffffu, ahead, 0);
                        it = item_of<kRows, KT, SPLIT, CROSS>(c, p, idx);
                    }
                } else {
                    it = item_of<kRows, KT, SPLIT, CROSS>(c, p, idx);
                }
                ok = warp_wait(&c.ite[nth % kItemRing], ((nth / kItemRing) & 1) ^ 1, &c.abort);
                if (!ok)
                    break;
                if (lane == 0) {
                    c.items[nth % kItemRing] = it;
                    if constexpr (CROSS)
                        c.parts[nth % kItemRing] = it;
                    mbar_arrive(&c.itf[nth % kItemRing]);
                }
                __syncwarp();
                if (over || it.t0 == it.t1)
                    continue;
                const long long unit = p.page_size
                                           ? static_cast<long long>(it.layer) * p.n_pages * p.n_kv_heads
                                           : static_cast<long long>(it.layer * p.batch + it.b) * p.n_kv_heads + it.kvh;
                // cache row of list block j (a box of 16 rows), -16 (rows of zeros) where there is none
                auto row_of = [&](int j) -> int {
                    if (j >= it.nb)
                        return -16;
                    const int pos = j * 16 + (j < it.sb ? 0 : it.base);
                    if (p.page_size == 0)
                        return static_cast<int>(unit * p.capacity + pos);
                    const int page = __ldg(p.page_table + static_cast<size_t>(it.b) * p.max_pages + (pos >> 4));
                    if (page < 0 || page >= p.n_pages) {
                        raise_error(p.err, 0x1u);  // SFI_DEVERR_PAGE_RANGE
                        return -16;
                    }
                    return static_cast<int>((unit + static_cast<long long>(page) * p.n_kv_heads + it.kvh) * 16);
                };
                // lane: block lane % kBlocks, 64-column half lane / kBlocks
                const int blk = lane % kBlocks, half = lane / kBlocks;
                int row = half < 2 ? row_of(it.t0 * kBlocks + blk) : 0;
                bool have_q = false;
                for (int t = it.t0; t < it.t1; ++t) {
                    const int st = use % ST, ph = (use / ST) & 1;
                    uint8_t *k = kv_smem + st * kStage, *v = k + 2 * kHalfKV;
                    const int here = row;
                    if (half < 2 && t + 1 < it.t1)
                        row = row_of((t + 1) * kBlocks + blk);
                    if (lane == 0) {
                        ok = mbar_wait(&c.ke[st], ph ^ 1, &c.abort);
                        if (ok)
                            mbar_arrive_expect_tx(&c.kf[st], 2 * kHalfKV);
                    }
                    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                    if (!ok)
                        break;
                    if (half < 2)
                        tma_load_2d(k + half * kHalfKV + blk * 2048, &tm_k, &c.kf[st], 64 * half, here);
                    if (!have_q && lane == 0) {
                        // the queries behind the first keys: they wait for the last item's scores
                        ok = mbar_wait(&c.qe, (items & 1) ^ 1, &c.abort);
                        if (ok) {
                            mbar_arrive_expect_tx(&c.qf, NQ * 2 * kHalfQ);
#pragma unroll
                            for (int a = 0; a < NQ; ++a)
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    tma_load_3d(smem + (2 * a + h) * kHalfQ, &tm_q, &c.qf, 64 * h, it.kvh * G,
                                                it.layer * p.n_rows + it.r0 + a * (QR / G));
                        }
                    }
                    if (!have_q) {
                        have_q = true;
                        if (__shfl_sync(0xffffffffu, ok ? 1 : 0, 0))
                            ++items;
                    }
                    if (lane == 0) {
                        ok = ok && mbar_wait(&c.ve[st], ph ^ 1, &c.abort);
                        mbar_arrive_expect_tx(&c.vf[st], ok ? 2 * kHalfKV : 0);
                    }
                    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                    if (ok && half < 2)
                        tma_load_2d(v + half * kHalfKV + blk * 2048, &tm_v, &c.vf[st], 64 * half, here);
                    __syncwarp();
                    ++use;
                    if (!ok)
                        break;
                }
            }
            if (lane == 0) {
                if (CROSS && !SPLIT) {
                    // the last CTA to be done with the queue leaves it as it was
                    __threadfence();
                    if (atomic_add_acq_rel_gpu(p.tickets + 1, 1) == static_cast<int>(gridDim.x) - 1) {
                        p.tickets[0] = 0;
                        p.tickets[1] = 0;
                    }
                }
                if (!ok)
                    wfail(c, p.err);
                // never leave a copy in flight into shared memory that is given up
                for (int j = max(0, use - ST); j < use; ++j) {
                    mbar_wait(&c.kf[j % ST], (j / ST) & 1, nullptr);
                    mbar_wait(&c.vf[j % ST], (j / ST) & 1, nullptr);
                }
                if (items > 0)
                    mbar_wait(&c.qf, (items - 1) & 1, nullptr);
            }
            __syncwarp();
        } else if (warp == 1) {
            // -------------------------------------------------------------------- MMA issuer
            // The whole warp runs this loop on values that are uniform over it (trip counts, stages,
            // the tensor-memory base), and one elected lane issues: the descriptors then live in
            // uniform registers, and an MMA costs two additions beside itself. Issued from one
            // lane's own branch an MMA took 85-95 clocks (for 32-64 of work): the tensor core
            // waited for its instructions.
            constexpr uint32_t idesc_s = idesc_bf16(128, KT, false, false);
            constexpr uint32_t idesc_o = idesc_bf16(128, 128, false, true);
            const uint64_t dq0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
            const uint64_t dk0 = smem_desc_sw128(smem_u32(kv_smem), 16, 1024);
            const uint64_t dv0 = smem_desc_sw128(smem_u32(kv_smem) + 2 * kHalfKV, kHalfKV, 1024);
            const uint32_t tm = uniform(tmem), all = uniform(total);
            uint32_t seq = 0, items = 0, nth = 0;     // tiles, items with tiles and items so far
            bool ok = true;
            // S of q tile A from the keys in stage st
            auto scores = [&](int A, uint32_t st, uint32_t buf) {
                const uint64_t dq = dq0 + A * (2 * kHalfQ / 16), dk = dk0 + st * (kStage / 16);
                const uint32_t d = tm + A * kQTile + buf * kSW;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    umma_bf16(d, dq + ((kk >> 2) * kHalfQ + (kk & 3) * 32) / 16,
                              dk + ((kk >> 2) * kHalfKV + (kk & 3) * 32) / 16, idesc_s, kk > 0 ? 1u : 0u);
                umma_commit(&c.sf[A][buf]);
            };
            auto products = [&](int A, uint32_t st, uint32_t buf, int half, bool first) {
                const uint64_t dv = dv0 + st * (kStage / 16);
                const uint32_t d = tm + A * kQTile + NS * kSW, w = tm + A * kQTile + buf * kSW;
#pragma unroll
                for (int part = 0; part < PARTS; ++part)
#pragma unroll
                    for (int k2 = 0; k2 < kBlocks / NH; ++k2) {
                        const int kk = half * (kBlocks / NH) + k2;
                        umma_bf16_ta(d, part == 2 ? w + KT + kk * 8 : w + (kk >> 1) * 32 + part * 16 + (kk & 1) * 8,
                                     dv + kk * 128,
                                     idesc_o,
                                     kk > 0 || part > 0 ? 1u : first ? 0u : 1u);
                    }
                if (half == NH - 1)
                    umma_commit(&c.od[A][buf]);
            };
            for (uint32_t idx = blockIdx.x; (kFed || idx < all) && ok; idx += gridDim.x) {
                Item<CROSS> it;
                ok = next_item(nth++, it);
                if (!ok || (kFed && it.np == 0))
                    break;
                const uint32_t end = seq + uniform(it.t1 - it.t0);
                if (seq == end)
                    continue;
                ok = warp_wait(&c.qf, items & 1, &c.abort);
                // Steps: the product of a tile and at once the scores that take over its buffer, NS tiles
                // ahead of the softmax; the first NS steps have no product yet. (One copy of this code:
                // with one of its own for an item's first scores, four 32K prompts under a window of 64
                // take 450 us, so 444.)
                const uint32_t begin = seq;
                for (uint32_t next = seq; next < end + NS && ok; ++next) {
                    const uint32_t st = seq % ST, buf = next % NS;
#pragma unroll
                    for (int A = 0; A < NQ; ++A) {
                        if (next >= begin + NS) {
#pragma unroll
                            for (int half = 0; half < NH; ++half) {
                                ok = ok && warp_poll([&] {
                                    return mbar_test_wait(&c.pf[A][NH == 2 ? half : buf], (seq / NS) & 1) &&
                                           (A > 0 || half > 0 || mbar_test_wait(&c.vr[st], (seq / ST) & 1)) &&
                                           (seq > begin || half > 0 || mbar_test_wait(&c.oe[A], (items & 1) ^ 1));
                                }, &c.abort);
                                if (!ok)
                                    break;
                                tc_fence_after();
                                if (elect_one()) {
                                    products(A, st, buf, half, F32 ? (seq - begin) % kFlush == 0 : seq == begin);
                                    if (A == NQ - 1 && half == NH - 1)
                                        umma_commit(&c.ve[st]);
                                }
                                __syncwarp();
                            }
                            if (!ok)
                                break;
                        }
                        if (next >= end)
                            continue;
                        // (asked only now: the product does not wait for keys that are on their way)
                        if (A == 0) {
                            ok = warp_poll([&] { return mbar_test_wait(&c.kf[next % ST], (next / ST) & 1); },
                                           &c.abort);
                            if (!ok)
                                break;
                            tc_fence_after();
                        }
                        if (elect_one()) {
                            scores(A, next % ST, buf);
                            if (A == NQ - 1) {
                                umma_commit(&c.ke[next % ST]);
                                if (next + 1 == end)
                                    umma_commit(&c.qe);
                            }
                        }
                        __syncwarp();
                    }
                    if (next >= begin + NS)
                        ++seq;
                }
                if (!ok)
                    break;
                ++items;
            }
            if (lane == 0 && !ok)
                wfail(c, p.err);
            if (elect_one())
                umma_commit(&c.drain);
            __syncwarp();
            mbar_wait(&c.drain, 0, nullptr);
            __syncwarp();
        } else if (warp == 2) {
            // ------------------------------------------------- V rows that nobody may see := 0
            int use = 0;
            uint32_t nth = 0;
            bool ok = true;
            for (int idx = blockIdx.x; (kFed || idx < total) && ok; idx += gridDim.x) {
                Item<CROSS> it;
                ok = next_item(nth++, it);
                if (!ok || (kFed && it.np == 0))
                    break;
                const int last = end_of(it) - 1;
                for (int t = it.t0; t < it.t1; ++t, ++use) {
                    const int st = use % ST;
                    ok = warp_wait(&c.vf[st], (use / ST) & 1, &c.abort);
                    if (!ok)
                        break;
                    uint8_t *v = kv_smem + st * kStage + 2 * kHalfKV;
                    bool wrote = false;
#pragma unroll
                    for (int i = 0; i < KT / 32; ++i) {
                        const int r = i * 32 + lane, col = t * KT + r, blk = col >> 4;
                        const int pos = col + (blk < it.sb ? 0 : it.base);
                        // (blocks behind the list were filled with zeros)
                        const bool seen = blk >= it.nb || (pos <= last && (CROSS || pos < p.n_sink || pos >= it.lo));
                        uint32_t m = __ballot_sync(0xffffffffu, !seen);
                        wrote = wrote || m != 0;
                        while (m) {
                            const int rr = i * 32 + __ffs(m) - 1;
                            m &= m - 1;
                            if (lane < 16)
                                reinterpret_cast<uint4 *>(v + (lane >> 3) * kHalfKV + rr * 128)[lane & 7] =
                                    make_uint4(0, 0, 0, 0);
                        }
                    }
                    if (wrote)
                        fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&c.vr[st]);
                }
            }
            if (!ok && lane == 0)
                wfail(c, p.err);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        tmem_dealloc(tmem, kCols);
    }
}

template <int NQ, int KT, int ST, int NS, int QR, int PARTS, bool F32, bool SPLIT, bool CROSS>
cudaError_t launch_one(const WindowParams &p, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                       const CUtensorMap &tm_q, int grid, cudaStream_t stream)
{
    auto *kern = window_kernel<NQ, KT, ST, NS, QR, PARTS, F32, SPLIT, CROSS>;
    constexpr int smem = window_smem<NQ, KT, ST, QR>();
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = launch_pdl(kern, dim3(grid), dim3(128 + 128 * NQ), smem, stream, tm_k, tm_v, tm_q, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool CROSS, int NQ, int KT, int ST, int NS, int QR, int PARTS, bool F32>
cudaError_t launch_form(const WindowParams &p, bool split, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                        const CUtensorMap &tm_q, int grid, cudaStream_t stream)
{
    return split ? launch_one<NQ, KT, ST, NS, QR, PARTS, F32, true, CROSS>(p, tm_k, tm_v, tm_q, grid, stream)
                 : launch_one<NQ, KT, ST, NS, QR, PARTS, F32, false, CROSS>(p, tm_k, tm_v, tm_q, grid, stream);
}

// The form for items of `rows` operand rows.
template <bool CROSS>
cudaError_t launch_rows(const WindowParams &p, int rows, bool split, const CUtensorMap &tm_k,
                        const CUtensorMap &tm_v, const CUtensorMap &tm_q, int grid, cudaStream_t stream)
{
    if (rows == 256)        // (bf16 outputs only)
        return launch_form<CROSS, 2, 128, 2, 1, 128, 1, false>(p, split, tm_k, tm_v, tm_q, grid, stream);
    if (rows == 16)
        return p.out_fp32 ? launch_form<CROSS, 1, 64, 4, 2, 16, 3, true>(p, split, tm_k, tm_v, tm_q, grid, stream)
                          : launch_form<CROSS, 1, 64, 3, 2, 16, 2, false>(p, split, tm_k, tm_v, tm_q, grid, stream);
    return p.out_fp32 ? launch_form<CROSS, 1, 64, 4, 2, 128, 3, true>(p, split, tm_k, tm_v, tm_q, grid, stream)
                      : launch_form<CROSS, 1, 64, 2, 2, 128, 1, false>(p, split, tm_k, tm_v, tm_q, grid, stream);
}

}  // namespace
}  // namespace sfi
