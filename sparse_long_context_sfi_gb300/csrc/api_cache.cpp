// api_cache.cpp -- the extern "C" entry points of include/sfi.h that keep the cache around the
// decode path: pages, prompt chunks and their attention, rotary positions, an encoder's states, beam
// search and log probabilities. Argument checks, workspace layout and launches; no allocation, no
// synchronisation.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstring>

#include "api_common.h"

using namespace sfi;

namespace {

bool misaligned256(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 255u) != 0; }

PageParams page_params(const sfi_kv_cache *kv, int32_t *table, int32_t *refs, const uint8_t *active)
{
    PageParams p;
    p.batch = kv->batch;
    p.n_kv_heads = kv->n_kv_heads;
    p.capacity = kv->capacity;
    p.page_size = kv->page_size;
    p.n_pages = kv->n_pages;
    p.max_pages = kv->max_pages_per_seq;
    p.max_len = kv->max_len;
    p.table = table;
    p.refs = refs;
    p.seq_len = kv->seq_len;
    p.active = active;
    p.err = kv->err;
    return p;
}

// The table is written through the pool, so it must be the one that the cache reads.
sfi_status check_pool(const sfi_kv_cache *kv, const sfi_page_pool *pool)
{
    const sfi_status st = check_kv(kv);
    if (st != SFI_OK)
        return st;
    if (kv->page_size == 0 || !pool || !pool->page_table || !pool->refs ||
        pool->page_table != kv->page_table)
        return SFI_ERR_INVALID_ARG;
    return SFI_OK;
}

size_t page_scratch(const sfi_kv_cache *kv, char *base, PageScratch *s)
{
    const size_t pages = static_cast<size_t>(kv->n_pages) * sizeof(int32_t);
    const int words = (kv->max_pages_per_seq + 31) / 32 + 1;   // a range may start inside a word
    size_t o = 0;
    auto take = [&](size_t bytes) {
        char *at = base + o;
        o = align256(o + bytes);
        return static_cast<void *>(at);
    };
    s->list = static_cast<int32_t *>(take(pages));
    s->movers = static_cast<int32_t *>(take(pages));
    s->rank = static_cast<int32_t *>(take(pages));
    s->n_moves = static_cast<int32_t *>(take(2 * sizeof(int32_t)));
    const size_t tasks = static_cast<size_t>(kv->batch) * words;
    s->marks = static_cast<uint32_t *>(take(tasks * sizeof(uint32_t)));
    s->counts = static_cast<int32_t *>(take((tasks + 1) * sizeof(int32_t)));
    s->copies = static_cast<int4 *>(take(static_cast<size_t>(kv->batch) * sizeof(int4)));
    return o;
}

sfi_status check_ws(void *ws, size_t ws_bytes, size_t need)
{
    return !ws || ws_bytes < need || misaligned256(ws) ? SFI_ERR_WORKSPACE : SFI_OK;
}

// Rows of a chunk: row_start NULL means one row per sequence.
sfi_status check_rows(const sfi_kv_cache *kv, const int32_t *row_start, int32_t n_rows,
                      int32_t max_rows)
{
    if (n_rows < 0 || max_rows < 0 || (!row_start && n_rows != kv->batch) ||
        (!row_start && max_rows < 1))
        return SFI_ERR_INVALID_ARG;
    if (1LL * n_rows * kv->n_q_heads * kv->n_layers >= (1LL << 31))
        return SFI_ERR_UNSUPPORTED;
    return SFI_OK;
}

// How sfi_window_attn runs with items of `rows` operand rows (16, 128 or 256).
struct WindowShape {
    int rows, slots;        // operand rows per item; CTAs that are resident at once
    long long items;        // bound of the items before splitting
    long long most_split;   // splits of an item that fill the slots
    int part_rows;
};

WindowShape window_shape(const sfi_kv_cache *kv, int n_rows, int max_rows, int rows, bool fp32)
{
    WindowShape s;
    const int g = kv->n_q_heads / kv->n_kv_heads, sms = sm_count();
    s.rows = rows;
    s.slots = rows == 256 || fp32 ? sms : 2 * sms;
    const long long seqs = n_rows < kv->batch ? n_rows : kv->batch;
    const long long units = 1LL * kv->n_kv_heads * kv->n_layers;
    s.items = (1LL * n_rows * g / s.rows + seqs) * units;
    long long likely = (1LL * n_rows * g + s.rows - 1) / s.rows;
    likely = (likely > seqs ? likely : seqs) * units;
    const long long split = likely > 0 ? s.slots / likely : 1;
    s.most_split = split < 1 ? 1 : split > 64 ? 64 : split;
    s.part_rows = static_cast<int>(1LL * max_rows * g < s.rows ? 1LL * max_rows * g : s.rows);
    return s;
}

// The item size. 16 rows hold a single token's heads and leave room for a third stage. Two q
// tiles (256 rows) halve the reads of K and V and keep the tensor core busy while the other
// tile is in its softmax, but only one such CTA fits an SM: where the reach of a row is short,
// an item is mostly start and end, which two CTAs of 128 rows overlap. Measured, us of 128 and of
// 256 rows: an 8K chunk of 32 heads, window 64: 37, 50; 256: 62, 64; 384: 77, 75; 512: 91, 86; 1024: 149,
// 130. Eight ragged paged prompts of 64 heads, 256: 129, 139; 384: 163, 160; 512: 197, 184; 1024: 334,
// 287. (The two meet between 256 and 384.) fp32 outputs take the tensor memory of a second q
// tile, and of a second CTA, for themselves.
int window_rows(const sfi_kv_cache *kv, int max_rows, int n_window, bool fp32)
{
    const long long all = 1LL * max_rows * (kv->n_q_heads / kv->n_kv_heads);
    const int reach = n_window < kv->max_len ? n_window : kv->max_len;
    return all <= 16 ? 16 : all > 128 && reach >= 512 && !fp32 ? 256 : 128;
}

// Sized for any item size and split, so that it holds for every max_len and window. The tickets
// come first and their room does not depend on the call, so that calls of other shapes on the
// same workspace find them as this one leaves them, zero: items are split only if at least two
// CTAs are left for each, and the bound of their number is at most twice the likely one, so no
// more are split than CTAs fit, two to an SM.
size_t window_scratch(const sfi_kv_cache *kv, int n_rows, int max_rows, char *base, WindowParams *p)
{
    size_t o = 0, parts = 1;
    for (int rows : {16, 128, 256}) {
        const WindowShape s = window_shape(kv, n_rows, max_rows, rows, false);
        const size_t m = s.most_split > 1 ? static_cast<size_t>(s.items) * s.most_split * s.part_rows : 1;
        parts = m > parts ? m : parts;
    }
    const int sms = sm_count();
    const size_t tickets = 2 * static_cast<size_t>(sms > 0 ? sms : 1);
    auto take = [&](size_t bytes) {
        char *at = base + o;
        o = align256(o + bytes);
        return static_cast<void *>(at);
    };
    p->tickets = static_cast<int *>(take(tickets * sizeof(int)));
    p->part_ml = static_cast<float2 *>(take(parts * sizeof(float2)));
    p->parts = static_cast<float *>(take(parts * kHeadDim * sizeof(float)));
    return o;
}

// The shape and the workspace of sfi_cross_attn, whose items are cut where the CTAs' equal shares of
// all key tiles end: two pieces to a CTA at most, and a ticket to a CTA.
size_t cross_scratch(const sfi_kv_cache *kv, int max_rows, char *base, WindowParams *p)
{
    const int g = kv->n_q_heads / kv->n_kv_heads, sms = sm_count() > 0 ? sm_count() : 1;
    const long long all = 1LL * max_rows * g;
    size_t o = 0, rows = 0;
    for (long long r : {16, 128, 256}) {
        const size_t n = static_cast<size_t>(all < r ? all : r) * 2 * (r == 256 ? sms : 2 * sms);
        rows = n > rows && (r == 16 || all > 16) ? n : rows;
    }
    auto take = [&](size_t bytes) {
        char *at = base + o;
        o = align256(o + bytes);
        return static_cast<void *>(at);
    };
    p->tickets = static_cast<int *>(take(2 * static_cast<size_t>(sms) * sizeof(int)));
    p->part_ml = static_cast<float2 *>(take(rows * sizeof(float2)));
    p->parts = static_cast<float *>(take(rows * kHeadDim * sizeof(float)));
    return o;
}

sfi_status check_beam(const sfi_beam *b)
{
    if (!b || b->n_groups < 1 || b->n_beams < 1 || b->vocab < 1 || b->row_stride < b->vocab ||
        b->eos >= b->vocab)
        return SFI_ERR_INVALID_ARG;
    if (b->n_beams > kMaxBeams || 1LL * b->n_groups * b->n_beams > 65535 ||
        1LL * b->vocab * b->n_beams > (1LL << 30))
        return SFI_ERR_UNSUPPORTED;
    return SFI_OK;
}

// CTAs per row: at most the four per SM that are resident at once, each of whose eight warps
// has a whole 512-token chunk or more.
int beam_splits(const sfi_beam *b)
{
    const int rows = b->n_groups * b->n_beams, sms = sm_count();
    int s = 4 * sms / rows;
    const int most = b->vocab / 4096 + 1;
    s = s < most ? s : most;
    return s < 1 ? 1 : s > 64 ? 64 : s;
}

size_t beam_scratch(const sfi_beam *b, char *base, BeamParams *p)
{
    const size_t rows = static_cast<size_t>(b->n_groups) * b->n_beams;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        char *at = base + o;
        o = align256(o + bytes);
        return static_cast<void *>(at);
    };
    p->splits = beam_splits(b);
    // (room for the most groups, so that calls of other shapes leave the tickets zero)
    p->tickets = static_cast<int *>(take(65536 * sizeof(int)));
    p->part_stat = static_cast<float2 *>(take(rows * p->splits * sizeof(float2)));
    p->part_x = static_cast<float *>(take(rows * p->splits * b->n_beams * sizeof(float)));
    p->part_v = static_cast<int32_t *>(take(rows * p->splits * b->n_beams * sizeof(int32_t)));
    return o;
}

sfi_status check_rope(const sfi_rope *r)
{
    if (!r || r->rot_dim < 2 || r->rot_dim > kHeadDim || (r->rot_dim & 1) || !std::isfinite(r->amplitude) ||
        !r->turns || (reinterpret_cast<uintptr_t>(r->turns) & 7u) || !aligned16(r->q_norm) || !aligned16(r->k_norm))
        return SFI_ERR_INVALID_ARG;
    if ((r->q_norm || r->k_norm) && !(r->norm_eps > 0.f && std::isfinite(r->norm_eps)))
        return SFI_ERR_INVALID_ARG;
    return SFI_OK;
}

// Rows of `heads` heads each; written in place only where they are packed.
bool rope_rows_ok(const void *in, int64_t stride, const void *out, int heads)
{
    const int64_t packed = static_cast<int64_t>(heads) * kHeadDim;
    return aligned16(in) && aligned16(out) && stride >= packed && stride % 8 == 0 &&
           (in != out || stride == packed);
}

sfi_status rope(bool append, const sfi_kv_cache *kv, const sfi_rope *r, const sfi_rope_rows *rows,
                const int32_t *row_start, int32_t n_rows, int32_t max_rows, const uint8_t *active,
                void *stream)
{
    sfi_status st = check_kv(kv);
    if (st != SFI_OK || (st = check_rope(r)) != SFI_OK ||
        (st = check_rows(kv, row_start, n_rows, max_rows)) != SFI_OK)
        return st;
    if (!rows || !rows->q != !rows->q_out || (append ? rows->k_out != nullptr : !rows->k != !rows->k_out))
        return SFI_ERR_INVALID_ARG;
    if (n_rows == 0)
        return SFI_OK;
    if (append ? !rows->k || !rows->v : !rows->q && !rows->k)
        return SFI_ERR_INVALID_ARG;
    if ((rows->q && !rope_rows_ok(rows->q, rows->q_stride, rows->q_out, kv->n_q_heads)) ||
        (rows->k && !rope_rows_ok(rows->k, rows->k_stride, rows->k_out, kv->n_kv_heads)) ||
        (append && !rope_rows_ok(rows->v, rows->v_stride, nullptr, kv->n_kv_heads)))
        return SFI_ERR_INVALID_ARG;
    RopeParams p;
    std::memset(&p, 0, sizeof p);
    p.c.pg = page_params(kv, const_cast<int32_t *>(kv->page_table), nullptr, active);
    p.c.row_start = row_start;
    p.c.n_rows = n_rows;
    p.c.max_rows = max_rows;
    p.n_layers = kv->n_layers;
    p.n_q_heads = kv->n_q_heads;
    p.q = rows->q;
    p.k = rows->k;
    p.q_stride = rows->q_stride;
    p.k_stride = rows->k_stride;
    p.q_out = rows->q_out;
    if (append) {
        p.v = rows->v;
        p.v_stride = rows->v_stride;
        p.k_cache = kv->k;
        p.v_cache = kv->v;
    } else {
        p.k_out = rows->k_out;
    }
    p.pos = rows->pos;
    p.rot = r->rot_dim;
    p.interleaved = r->interleaved ? 1 : 0;
    p.amplitude = r->amplitude;
    p.eps = r->norm_eps;
    p.turns = r->turns;
    p.q_norm = r->q_norm;
    p.k_norm = r->k_norm;
    const int sms = sm_count();
    if (sms <= 0)
        return SFI_ERR_CUDA;
    return launch_status(launch_rope(p, sms, as_stream(stream)));
}

// sfi_window_attn, or with `cross` rows that see all of their sequence (n_sink 0, n_window INT_MAX).
sfi_status attend(bool cross, const sfi_kv_cache *kv, const void *q, void *out, int32_t out_fp32,
                  const int32_t *row_start, int32_t n_rows, int32_t max_rows, int32_t n_sink,
                  int32_t n_window, const uint8_t *active, void *ws, size_t ws_bytes, void *stream)
{
    sfi_status st = check_kv(kv);
    if (st != SFI_OK)
        return st;
    if (n_sink < 0 || n_window < 1)
        return SFI_ERR_INVALID_ARG;
    if ((st = check_rows(kv, row_start, n_rows, max_rows)) != SFI_OK)
        return st;
    WindowParams p;
    std::memset(&p, 0, sizeof p);
    const size_t need = cross ? cross_scratch(kv, max_rows, static_cast<char *>(ws), &p)
                              : window_scratch(kv, n_rows, max_rows, static_cast<char *>(ws), &p);
    if ((st = check_ws(ws, ws_bytes, need)) != SFI_OK)
        return st;
    if (n_rows == 0 || max_rows == 0)
        return SFI_OK;
    if (!q || !out || !aligned16(q) || !aligned16(out))
        return SFI_ERR_INVALID_ARG;
    const bool fp32 = out_fp32 != 0;
    const int rows = window_rows(kv, max_rows, n_window, fp32);
    CUtensorMap tk, tv, tq;
    if (!make_map(&tk, kv->k, cache_rows(kv), 16u) || !make_map(&tv, kv->v, cache_rows(kv), 16u) ||
        !make_chunk_map(&tq, q, static_cast<uint64_t>(kv->n_layers) * n_rows,
                        static_cast<uint32_t>(kv->n_q_heads),
                        static_cast<uint32_t>(kv->n_q_heads / kv->n_kv_heads), rows == 16 ? 16u : 128u))
        return SFI_ERR_CUDA;
    p.n_layers = kv->n_layers;
    p.batch = kv->batch;
    p.n_kv_heads = kv->n_kv_heads;
    p.group = kv->n_q_heads / kv->n_kv_heads;
    p.group_log2 = p.group == 8 ? 3 : p.group == 4 ? 2 : p.group == 2 ? 1 : 0;
    p.heads_log2 = -1;
    for (int i = 0; i < 31; ++i)
        if (kv->n_kv_heads == 1 << i)
            p.heads_log2 = i;
    p.capacity = kv->capacity;
    p.page_size = kv->page_size;
    p.n_pages = kv->n_pages;
    p.max_pages = kv->max_pages_per_seq;
    p.max_len = kv->max_len;
    p.page_table = kv->page_table;
    p.seq_len = kv->seq_len;
    p.active = active;
    p.row_start = row_start;
    p.n_rows = n_rows;
    p.max_rows = max_rows;
    p.n_sink = n_sink;
    p.n_window = n_window;
    p.out = out;
    p.out_fp32 = out_fp32 ? 1 : 0;
    p.out_aligned32 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
    p.err = kv->err;
    const long long len = kv->max_len, reach = n_window < len ? n_window : len;
    const WindowShape s = window_shape(kv, n_rows, max_rows, rows, fp32);
    const int kt = rows == 256 ? 128 : 64;
    p.scale_log2 = static_cast<float>(1.4426950408889634074 / std::sqrt(static_cast<double>(kHeadDim)));
    p.part_rows = s.part_rows;
    if (cross) {
        // Few items are shared out by their key tiles, many taken whole from a queue, which leaves
        // the CTAs close together in the keys and joins nothing. Measured, us, shares and queue: 32 x 4 rows
        // of 1000 to 4001 keys (0.8 items a CTA) 61, 86; 300 rows of 8192 keys (0.5) 62, 114; 2048 (1.7) 214,
        // 222; ragged prompts of up to 701 rows of 0 to 1601 keys (5) 128, 95; 4 x 2048 of 8192 (6.7) 837, 761.
        // A share has at least as many tiles as join well: one row of 601 keys with 1, 2, 4 tiles 14, 14,
        // 17; of 8192 keys 31, 28, 22. (Key tiles of one unit are counted in 31 bits.)
        const double tiles = std::ceil(static_cast<double>(len) / kt);
        const double unit = (1. * n_rows * p.group / rows + kv->batch) * (tiles + 2.);
        const bool shares = s.items < 2 * s.slots && unit < 2147483647.;
        const double least = std::sqrt(tiles / 4.);
        p.n_split = !shares ? 1 : least > 2. ? static_cast<int>(least + 0.5) : 2;
        return launch_status(launch_cross(p, rows, shares, tk, tv, tq, s.slots, as_stream(stream)));
    }
    // Fewer items than CTAs that fit: split their keys, four tiles at least to a split.
    const long long span = reach + rows / p.group < len ? reach + rows / p.group : len;
    const long long tiles = (span + n_sink + 32 + kt - 1) / kt;
    long long split = s.most_split < tiles / 4 ? s.most_split : tiles / 4;
    split = split < 1 ? 1 : split;
    p.n_split = static_cast<int>(split);
    const long long all = s.items * split;
    const int grid = static_cast<int>(all < s.slots ? all : s.slots);
    return launch_status(launch_window(p, rows, tk, tv, tq, grid, as_stream(stream)));
}

sfi_status check_scoring(const sfi_scoring *s)
{
    if (!s || s->n_rows < 0 || s->vocab < 1 || s->row_stride < s->vocab || s->n_top < 0 || s->n_top > s->vocab)
        return SFI_ERR_INVALID_ARG;
    if (s->n_top > kMaxTop || s->vocab > (1 << 30) || s->n_rows > (1 << 30))
        return SFI_ERR_UNSUPPORTED;
    return SFI_OK;
}

// CTAs of a row and warps of a CTA: the least sum over the waves of CTAs (32 warps to an SM, 28 of the
// form with rank and entropy) of a warp's chunks (of 2 KB) and what a row's end costs in such steps: more
// with a list, for each token of it, for lanes of which three chunks hold one of them, so that all of
// theirs are read again (of k tokens in n lanes about k^3 / 6 n^2), and where CTAs are joined. Measured,
// us: 8192 rows of 32000 bf16 with rank and entropy, 1, 2, 4, 8 warps: no list 90, 91, 92, 114; 3 tokens
// 100, 108, 117, 176; 20 tokens 150, 126, 138, 224; 8192 rows of 1000, 3 tokens: 23, 35, 49, 113; 2048 of
// 128001, 8 tokens: 151, 99, 101, 125. 256 rows of 128001 fp32 with 20 tokens, 4 warps, 2, 3 and 4 CTAs a
// row: 41, 36, 35; 8 warps, 1, 2, 4: 39, 53, 55; 100 rows, 2 warps and 21 CTAs 29, 8 warps and 3 25.
void score_shape(const sfi_scoring *s, int sms, ScoreParams *p)
{
    const double of = s->logits_fp32 ? 512. : 1024., k = s->n_top;
    const double chunks = std::ceil(s->vocab / of), rows = s->n_rows > 0 ? s->n_rows : 1;
    double best = -1.;
    const double room = s->rank && s->entropy ? 28. : 32.;
    p->splits = 1;
    p->warps = 8;
    for (int warps = 8; warps >= 1; warps /= 2) {
        for (int splits = 1; splits <= 64 && (splits == 1 || (rows <= kMaxSplitRows && splits * warps <= chunks)); ++splits) {
            const double waves = std::ceil(rows * splits / (std::floor(room / warps) * (sms > 0 ? sms : 1)));
            const double steps = std::ceil(chunks / (warps * splits));
            const double again = steps * k * k * k / (17000. * warps * warps);
            const double cost = waves * (steps + again + (k > 0 ? 2.5 + k / 7. : 1.) + (splits > 1 ? 4. + k * splits / 40. : 0.));
            if (best < 0. || cost < best) {
                best = cost;
                p->splits = splits;
                p->warps = warps;
            }
        }
    }
}

size_t score_scratch(const sfi_scoring *s, char *base, ScoreParams *p)
{
    const int sms = sm_count();
    size_t o = 0;
    auto take = [&](size_t bytes) {
        char *at = base + o;
        o = align256(o + bytes);
        return static_cast<void *>(at);
    };
    score_shape(s, sms, p);
    const size_t parts = p->splits > 1 ? static_cast<size_t>(s->n_rows) * p->splits : 0;
    // (room that does not depend on the call, so that calls of other shapes leave the tickets zero)
    p->tickets = static_cast<int *>(take(kMaxSplitRows * sizeof(int)));
    p->part = static_cast<float4 *>(take(parts * sizeof(float4)));
    p->part_x = static_cast<float *>(take(parts * s->n_top * sizeof(float)));
    p->part_v = static_cast<int32_t *>(take(parts * s->n_top * sizeof(int32_t)));
    return o;
}

}  // namespace

extern "C" {

size_t sfi_pages_workspace_bytes(const sfi_kv_cache *kv)
{
    if (check_kv(kv) != SFI_OK || kv->page_size == 0)
        return 0;
    PageScratch s;
    return page_scratch(kv, nullptr, &s);
}

sfi_status sfi_pages_reserve(const sfi_kv_cache *kv, const sfi_page_pool *pool,
                             const int32_t *n_new, const uint8_t *active, uint8_t *ok, void *ws,
                             size_t ws_bytes, void *stream)
{
    sfi_status st = check_pool(kv, pool);
    if (st != SFI_OK)
        return st;
    PageScratch s;
    if ((st = check_ws(ws, ws_bytes, page_scratch(kv, static_cast<char *>(ws), &s))) != SFI_OK)
        return st;
    return launch_status(launch_reserve(page_params(kv, pool->page_table, pool->refs, active), n_new,
                                        ok, s, kv->k, kv->v, kv->n_layers, as_stream(stream)));
}

sfi_status sfi_pages_release(const sfi_kv_cache *kv, const sfi_page_pool *pool,
                             const uint8_t *active, void *stream)
{
    const sfi_status st = check_pool(kv, pool);
    if (st != SFI_OK)
        return st;
    return launch_status(launch_drop_pages(page_params(kv, pool->page_table, pool->refs, active), 0,
                                           0, 0, as_stream(stream)));
}

sfi_status sfi_pages_evict(const sfi_kv_cache *kv, const sfi_page_pool *pool, int32_t n_sink,
                           int32_t n_window, const uint8_t *active, void *stream)
{
    const sfi_status st = check_pool(kv, pool);
    if (st != SFI_OK)
        return st;
    if (n_sink < 0 || n_window < 1)
        return SFI_ERR_INVALID_ARG;
    return launch_status(launch_drop_pages(page_params(kv, pool->page_table, pool->refs, active), 1,
                                           n_sink, n_window, as_stream(stream)));
}

sfi_status sfi_pages_compact(const sfi_kv_cache *kv, const sfi_page_pool *pool, int32_t *n_used,
                             void *ws, size_t ws_bytes, void *stream)
{
    sfi_status st = check_pool(kv, pool);
    if (st != SFI_OK)
        return st;
    if (!n_used)
        return SFI_ERR_INVALID_ARG;
    PageScratch s;
    if ((st = check_ws(ws, ws_bytes, page_scratch(kv, static_cast<char *>(ws), &s))) != SFI_OK)
        return st;
    const int sms = sm_count();
    if (sms <= 0)
        return SFI_ERR_CUDA;
    return launch_status(launch_pages_compact(page_params(kv, pool->page_table, pool->refs, nullptr),
                                              n_used, s, kv->k, kv->v, kv->n_layers, sms * 8,
                                              as_stream(stream)));
}

sfi_status sfi_append_chunk(const sfi_kv_cache *kv, const void *k_new, const void *v_new,
                            const int32_t *row_start, int32_t n_rows, int32_t max_rows,
                            const uint8_t *active, void *stream)
{
    sfi_status st = check_kv(kv);
    if (st != SFI_OK)
        return st;
    if ((st = check_rows(kv, row_start, n_rows, max_rows)) != SFI_OK)
        return st;
    if (n_rows == 0)
        return SFI_OK;
    if (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new))
        return SFI_ERR_INVALID_ARG;
    ChunkParams p;
    p.pg = page_params(kv, const_cast<int32_t *>(kv->page_table), nullptr, active);
    p.row_start = row_start;
    p.n_rows = n_rows;
    p.max_rows = max_rows;
    return launch_status(launch_append_chunk(p, k_new, v_new, kv->k, kv->v, kv->n_layers,
                                             as_stream(stream)));
}

size_t sfi_window_workspace_bytes(const sfi_kv_cache *kv, int32_t n_rows, int32_t max_rows,
                                  int32_t n_sink, int32_t n_window)
{
    if (check_kv(kv) != SFI_OK || n_rows < 0 || max_rows < 0 || n_sink < 0 || n_window < 1)
        return 0;
    WindowParams p;
    return window_scratch(kv, n_rows, max_rows, nullptr, &p);
}

sfi_status sfi_window_attn(const sfi_kv_cache *kv, const void *q, void *out, int32_t out_fp32,
                           const int32_t *row_start, int32_t n_rows, int32_t max_rows,
                           int32_t n_sink, int32_t n_window, const uint8_t *active, void *ws,
                           size_t ws_bytes, void *stream)
{
    return attend(false, kv, q, out, out_fp32, row_start, n_rows, max_rows, n_sink, n_window, active, ws,
                  ws_bytes, stream);
}

size_t sfi_cross_workspace_bytes(const sfi_kv_cache *kv, int32_t n_rows, int32_t max_rows)
{
    if (check_kv(kv) != SFI_OK || n_rows < 0 || max_rows < 0)
        return 0;
    WindowParams p;
    return cross_scratch(kv, max_rows, nullptr, &p);
}

sfi_status sfi_cross_attn(const sfi_kv_cache *kv, const void *q, void *out, int32_t out_fp32,
                          const int32_t *row_start, int32_t n_rows, int32_t max_rows,
                          const uint8_t *active, void *ws, size_t ws_bytes, void *stream)
{
    return attend(true, kv, q, out, out_fp32, row_start, n_rows, max_rows, 0, INT_MAX, active, ws, ws_bytes,
                  stream);
}

sfi_status sfi_rope_turns(int32_t rot_dim, const sfi_rope_scaling *sc, uint64_t *turns, float *amplitude)
{
    if (rot_dim < 2 || rot_dim > kHeadDim || (rot_dim & 1) || !sc || !turns || !amplitude || sc->reserved != 0 ||
        sc->kind < SFI_ROPE_PLAIN || sc->kind > SFI_ROPE_SMOOTH)
        return SFI_ERR_INVALID_ARG;
    const bool stretched = sc->kind != SFI_ROPE_PLAIN;
    const bool parts = sc->kind == SFI_ROPE_RAMP || sc->kind == SFI_ROPE_SMOOTH;
    if (!(sc->base > 1.) || !std::isfinite(sc->base) ||
        (stretched && (!(sc->factor >= 1.) || !std::isfinite(sc->factor))) ||
        (parts && (!(sc->original_len > 0.) || !std::isfinite(sc->original_len) || !(sc->low > 0.) ||
                   !(sc->high > sc->low) || !std::isfinite(sc->high))) ||
        (sc->kind == SFI_ROPE_BASE && rot_dim == 2))
        return SFI_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    double base = sc->base, first = 0., last = 0.;
    if (sc->kind == SFI_ROPE_BASE)
        base *= std::pow(sc->factor, rot_dim / (rot_dim - 2.));
    if (sc->kind == SFI_ROPE_RAMP) {
        auto dim = [&](double t) { return rot_dim * std::log(sc->original_len / (two_pi * t)) / (2. * std::log(base)); };
        first = std::fmax(0., std::floor(dim(sc->high)));
        last = std::fmin(rot_dim - 1., std::ceil(dim(sc->low)));
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2. * i / rot_dim);
        double keep = 1.;       // the share that is not divided by the factor
        if (sc->kind == SFI_ROPE_LINEAR)
            keep = 0.;
        else if (sc->kind == SFI_ROPE_RAMP)
            keep = 1. - std::fmin(1., std::fmax(0., (i - first) / std::fmax(last - first, 0.001)));
        else if (sc->kind == SFI_ROPE_SMOOTH)
            keep = std::fmin(1., std::fmax(0., (sc->original_len * f / two_pi - sc->low) / (sc->high - sc->low)));
        if (keep < 1.)
            f = f * keep + f / sc->factor * (1. - keep);
        // (f <= 1, so below 2^64 units)
        turns[i] = static_cast<uint64_t>(std::floor(std::ldexp(f / two_pi, 64) + 0.5));
    }
    *amplitude = sc->kind == SFI_ROPE_RAMP ? static_cast<float>(0.1 * std::log(sc->factor) + 1.) : 1.f;
    return SFI_OK;
}

sfi_status sfi_rope_apply(const sfi_kv_cache *kv, const sfi_rope *r, const sfi_rope_rows *rows,
                          const int32_t *row_start, int32_t n_rows, int32_t max_rows,
                          const uint8_t *active, void *stream)
{
    return rope(false, kv, r, rows, row_start, n_rows, max_rows, active, stream);
}

sfi_status sfi_rope_append(const sfi_kv_cache *kv, const sfi_rope *r, const sfi_rope_rows *rows,
                           const int32_t *row_start, int32_t n_rows, int32_t max_rows,
                           const uint8_t *active, void *stream)
{
    return rope(true, kv, r, rows, row_start, n_rows, max_rows, active, stream);
}

sfi_status sfi_reorder(const sfi_kv_cache *kv, const sfi_page_pool *pool,
                       const sfi_budget *budget, const sfi_sparse_mem *mem, const int32_t *src,
                       void *stream)
{
    sfi_status st = kv && kv->page_size ? check_pool(kv, pool) : check_kv(kv);
    if (st != SFI_OK)
        return st;
    if (!src || (kv->page_size == 0 && pool))
        return SFI_ERR_INVALID_ARG;
    if (mem) {
        if ((st = check_budget(budget)) != SFI_OK)
            return st;
        if (!mem->kc || !mem->vc || !mem->sel_cnt || !mem->rows || !aligned16(mem->kc) ||
            !aligned16(mem->vc) || (budget->n_select > 0 && !mem->sel_idx))
            return SFI_ERR_INVALID_ARG;
    }
    ReorderParams p;
    std::memset(&p, 0, sizeof p);
    p.batch = kv->batch;
    p.n_kv_heads = kv->n_kv_heads;
    p.n_pages = kv->n_pages;
    p.src = src;
    p.err = kv->err;
    auto part = [&](int i, int32_t *data, int layers, int cols, int32_t *refs) {
        p.ints[i].data = data;
        p.ints[i].cols = cols;
        p.ints[i].slices = layers * ((cols + 31) / 32);
        p.ints[i].refs = refs;
    };
    if (pool)
        part(0, pool->page_table, 1, kv->max_pages_per_seq, pool->refs);
    if (mem) {
        if (budget->n_select > 0)
            part(1, mem->sel_idx, kv->n_layers, kv->n_kv_heads * budget->n_select, nullptr);
        part(2, mem->sel_cnt, kv->n_layers, kv->n_kv_heads, nullptr);
        part(3, mem->rows, kv->n_layers, kv->n_kv_heads, nullptr);
    }
    part(4, kv->seq_len, 1, 1, nullptr);
    // the rows first: the matrices say how many rows there are
    cudaError_t e = cudaSuccess;
    if (mem)
        e = launch_reorder_rows(p, mem->kc, mem->vc, kv->n_layers, budget->n_sink + budget->n_select,
                                mem->rows, 1, as_stream(stream));
    if (e == cudaSuccess && kv->page_size == 0)
        e = launch_reorder_rows(p, kv->k, kv->v, kv->n_layers, kv->capacity, kv->seq_len, 0,
                                as_stream(stream));
    if (e == cudaSuccess)
        e = launch_reorder_ints(p, as_stream(stream));
    return launch_status(e);
}

size_t sfi_beam_workspace_bytes(const sfi_beam *beam)
{
    if (check_beam(beam) != SFI_OK)
        return 0;
    BeamParams p;
    return beam_scratch(beam, nullptr, &p);
}

sfi_status sfi_beam_select(const sfi_beam *beam, void *ws, size_t ws_bytes, void *stream)
{
    sfi_status st = check_beam(beam);
    if (st != SFI_OK)
        return st;
    if (!beam->logits || !beam->cum || !beam->parent || !beam->token || !beam->cum_out ||
        (beam->done && beam->eos < 0) ||
        (reinterpret_cast<uintptr_t>(beam->logits) & (beam->logits_fp32 ? 3u : 1u)))
        return SFI_ERR_INVALID_ARG;
    BeamParams p;
    std::memset(&p, 0, sizeof p);
    if ((st = check_ws(ws, ws_bytes, beam_scratch(beam, static_cast<char *>(ws), &p))) != SFI_OK)
        return st;
    p.n_groups = beam->n_groups;
    p.n_beams = beam->n_beams;
    p.vocab = beam->vocab;
    p.logits_fp32 = beam->logits_fp32 ? 1 : 0;
    p.eos = beam->eos < 0 ? -1 : beam->eos;
    p.row_stride = beam->row_stride;
    p.logits = beam->logits;
    p.cum = beam->cum;
    p.done = beam->done;
    p.rank_scale = beam->rank_scale;
    p.parent = beam->parent;
    p.token = beam->token;
    p.cum_out = beam->cum_out;
    p.done_out = beam->done_out;
    return launch_status(launch_beam_select(p, as_stream(stream)));
}

size_t sfi_scoring_workspace_bytes(const sfi_scoring *scoring)
{
    if (check_scoring(scoring) != SFI_OK)
        return 0;
    ScoreParams p;
    return score_scratch(scoring, nullptr, &p);
}

sfi_status sfi_score_tokens(const sfi_scoring *sc, void *ws, size_t ws_bytes, void *stream)
{
    sfi_status st = check_scoring(sc);
    if (st != SFI_OK)
        return st;
    if ((!sc->token && (sc->logprob || sc->rank)) || (sc->n_top > 0 && (!sc->top_token || !sc->top_logprob)) ||
        (sc->n_top == 0 && !sc->logprob && !sc->rank && !sc->entropy))
        return SFI_ERR_INVALID_ARG;
    ScoreParams p;
    std::memset(&p, 0, sizeof p);
    if ((st = check_ws(ws, ws_bytes, score_scratch(sc, static_cast<char *>(ws), &p))) != SFI_OK)
        return st;
    if (sc->n_rows == 0)
        return SFI_OK;
    if (!sc->logits || (reinterpret_cast<uintptr_t>(sc->logits) & (sc->logits_fp32 ? 3u : 1u)))
        return SFI_ERR_INVALID_ARG;
    p.n_rows = sc->n_rows;
    p.vocab = sc->vocab;
    p.logits_fp32 = sc->logits_fp32 ? 1 : 0;
    p.n_top = sc->n_top;
    p.row_stride = sc->row_stride;
    p.logits = sc->logits;
    p.token = sc->token;
    p.logprob = sc->logprob;
    p.rank = sc->rank;
    p.entropy = sc->entropy;
    p.top_token = sc->top_token;
    p.top_logprob = sc->top_logprob;
    return launch_status(launch_score(p, as_stream(stream)));
}

}  // extern "C"
