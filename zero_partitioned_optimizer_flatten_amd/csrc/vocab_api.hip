// Host side of the vocabulary operators: argument checks, workspace sizes and
// dispatch. The C ABI is declared and documented in include/zero.h.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/zero.h"
#include "vocab_internal.h"

namespace {

using zk::CaptureScope;
using zk::check_range;
using zk::fail;
using zk::hip_fail;

bool valid_dtype(zero_dtype d) { return d == ZERO_F32 || d == ZERO_BF16; }
int64_t dtype_size(zero_dtype d) { return d == ZERO_BF16 ? 2 : 4; }

// Rows are addressed by 32-bit offsets inside a tile of 256 of them.
constexpr int64_t kMaxRowBytes = (int64_t)1 << 22;
constexpr int64_t kMaxPiece = (int64_t)1 << 20;
// A dispatch holds fewer than 2^32 work-items.
constexpr int64_t kMaxUnits = 0xFFFFFF00ll;
constexpr int64_t kMaxInt = 0x7FFFFFFF;
constexpr int64_t kMaxRows = (int64_t)1 << 30, kMaxElements = (int64_t)1 << 42;

int64_t ceil_div(int64_t a, int64_t b) { return a / b + (a % b != 0); }

// A buffer of count elements of `size` bytes: there, aligned, long enough.
int check_buffer(const void *p, int64_t count, int64_t size, const char *what) {
    if (count == 0) return ZERO_OK;
    if (!p) return fail(ZERO_EINVAL, "%s is null", what);
    if ((uintptr_t)p % (uintptr_t)size)
        return fail(ZERO_EINVAL, "%s is not %lld-byte aligned", what, (long long)size);
    return check_range(p, count * size, what);
}

int check_ids(const void *ids, int32_t id_bytes, int64_t count, const char *what) {
    if (id_bytes != 4 && id_bytes != 8)
        return fail(ZERO_EINVAL, "%s: ids have 4 or 8 bytes (got %d)", what, id_bytes);
    return check_buffer(ids, count, id_bytes, what);
}

int check_table(int64_t rows, int64_t width, const char *what) {
    if (rows < 1 || width < 1)
        return fail(ZERO_EINVAL, "%s must have rows and columns (got %lld x %lld)", what, (long long)rows,
                    (long long)width);
    if (rows > kMaxRows || width > kMaxRows || rows > kMaxElements / width)
        return fail(ZERO_EUNSUPPORTED, "%s of %lld x %lld: more than 2^30 rows or columns, or 2^42 elements", what,
                    (long long)rows, (long long)width);
    return ZERO_OK;
}

int check_count(int64_t count, int64_t width) {
    if (count < 0) return fail(ZERO_EINVAL, "count must be >= 0 (got %lld)", (long long)count);
    if (count > kMaxInt || count * ceil_div(width, 4) > kMaxUnits)
        return fail(ZERO_EUNSUPPORTED, "%lld rows of %lld elements are more than one call takes", (long long)count,
                    (long long)width);
    return ZERO_OK;
}

// Whether the `na` bytes at a and the `nb` bytes at b meet.
bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && na > 0 && nb > 0 && x < y + (uint64_t)nb && y < x + (uint64_t)na;
}

int check_drop(const zero_drop *d, zk::Drop *out) {
    *out = {};
    out->scale = 1.0f;
    if (!d) return ZERO_OK;
    if (!(d->p >= 0.0 && d->p <= 1.0)) return fail(ZERO_EINVAL, "dropout: p must be in [0, 1] (got %g)", d->p);
    const int rc = d->counter ? check_buffer(d->counter, 1, 8, "dropout counter") : ZERO_OK;
    if (rc) return rc;
    out->key0 = (uint32_t)d->seed;
    out->key1 = (uint32_t)(d->seed >> 32);
    out->limit = (uint32_t)std::floor(d->p * 65536.0 + 0.5);
    out->scale = out->limit < 65536 ? (float)(65536.0 / (double)(65536 - out->limit)) : 0.0f;
    out->offset = d->offset;
    out->counter = d->counter;
    return ZERO_OK;
}

// Whether `bytes` bytes at p hold dropout's counter, which every workgroup reads.
bool holds_counter(const void *p, int64_t bytes, const zero_drop *d) { return d && overlap(p, bytes, d->counter, 8); }

int check_scale(double scale) {
    if (!std::isfinite((float)scale)) return fail(ZERO_EINVAL, "scale must be finite in fp32 (got %g)", scale);
    return ZERO_OK;
}

int check_workspace(const void *workspace, int64_t have, int64_t need) {
    if (have < need)
        return fail(ZERO_EINVAL, "workspace has %lld bytes, the call needs %lld", (long long)have, (long long)need);
    if (!workspace) return fail(ZERO_EINVAL, "workspace is null");
    if ((uintptr_t)workspace % 256) return fail(ZERO_EINVAL, "workspace is not 256-byte aligned");
    return check_range(workspace, need, "workspace");
}

int head_sizes(int64_t count, int64_t vocab, int64_t width, zero_dtype dtype, int64_t piece) {
    int rc = check_table(vocab, width, "table");
    if (rc) return rc;
    if (!valid_dtype(dtype)) return fail(ZERO_EINVAL, "unknown dtype %d", (int)dtype);
    if (count < 0) return fail(ZERO_EINVAL, "count must be >= 0 (got %lld)", (long long)count);
    if (count > kMaxInt) return fail(ZERO_EUNSUPPORTED, "%lld rows are more than one call takes", (long long)count);
    if (piece < 0) return fail(ZERO_EINVAL, "piece_rows must be >= 0 (got %lld)", (long long)piece);
    const int64_t es = dtype_size(dtype);
    if ((vocab + 128) * es > kMaxRowBytes || (width + 64) * es > kMaxRowBytes)
        return fail(ZERO_EUNSUPPORTED, "table of %lld x %lld: a row of either length must stay under 4 MiB",
                    (long long)vocab, (long long)width);
    if (piece > kMaxPiece && count > kMaxPiece)
        return fail(ZERO_EUNSUPPORTED, "pieces of %lld rows: at most 2^20", (long long)piece);
    // numbers of a piece against the vocabulary are turned 16 bytes to a work-item
    const int64_t rows = piece > 0 && piece < count ? piece : count;
    if (piece > 0 && (rows + 63) / 64 * 64 > kMaxUnits / 256 / ceil_div((vocab + 128) * es, 4096))
        return fail(ZERO_EUNSUPPORTED, "pieces of %lld rows take more than 64 GiB with a vocabulary of %lld", (long long)piece,
                    (long long)vocab);
    return ZERO_OK;
}

// The sort's workgroups read every id each: at most so many in all, about 5 s of them.
constexpr int64_t kMaxSortReads = (int64_t)1 << 42;

int check_sort(const zk::EmbedGradPlan &p, int64_t count, int64_t rows) {
    if (count > kMaxSortReads >> p.sort_groups_log2)
        return fail(ZERO_EUNSUPPORTED, "%lld ids of a table of %lld rows are more than one call takes", (long long)count,
                    (long long)rows);
    return ZERO_OK;
}

}  // namespace

namespace zk {

EmbedGradPlan plan_embed_grad(int64_t count, int64_t rows, int64_t width) {
    EmbedGradPlan p;
    // One workgroup to a compute unit, and more for tables of more than 131072 rows. Each
    // reads every token, up to 0.9e12 a second in all: 32768 tokens (64 columns) take 32 us
    // of 131072 rows, 43 of 2^18 and 115 of 2^20 with 2048 workgroups, 2^20 tokens of 2^20
    // rows 2.6 ms. check_sort() refuses what would take the device for long.
    p.sort_groups_log2 = 8;
    while (ceil_div(rows, (int64_t)1 << p.sort_groups_log2) > kSortIds) ++p.sort_groups_log2;
    p.ids_per_group = (int)ceil_div(rows, (int64_t)1 << p.sort_groups_log2);
    // About 4096 waves, and 8 to 256 tokens to each: enough to keep loads on their way,
    // few partial rows. 65536 tokens of 768 columns take 79 us (half the waves 86, a
    // quarter 109), 16384 of 4096 102 (twice the waves 107, four times 113; fp32 200,
    // twice the waves 194). Few tokens have a workgroup for each run, and no joining
    // follows (span 1).
    const int64_t chunks = ceil_div(width, kSpanCols), span = ceil_div(count * chunks, 4096);
    const bool runs = count <= kRunTokens && count * chunks < (int64_t)1 << 22;     // a dispatch's limit
    p.span = runs ? 1 : (int)(span < 8 ? 8 : span > 256 ? 256 : span);
    p.spans = ceil_div(count, p.span);
    const int64_t pitch = chunks * kSpanCols;
    p.count_off = 0;
    p.sorted_off = 256;
    p.partial_off = p.sorted_off + ceil_div(count * (int64_t)sizeof(SortedToken), 256) * 256;
    p.bytes = p.partial_off + (p.spans > 1 && p.span > 1 ? 2 * p.spans * pitch * (int64_t)sizeof(float) : 0);
    return p;
}

namespace {

int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

constexpr int64_t kMaxSlots = 1024;

// The tile that takes least time: rounds of as many tiles as run at once, by the
// stages of a tile and what its epilogue takes, with a last round cut into parts as
// the kernels' schedule does. A stage of a round takes 1, 0.62 and 0.6 by the tile
// (bf16): the middle and the small tile multiply at 0.8 and 0.3 of the large one's
// rate, since they bring 2 and 2.5 times as much to LDS for it (2048 rows of GPT-2's
// head: 665 us with large tiles, 704 with middle, 1105 with small). With fp32 the
// matrix cores bound all three (8192 x 32000 x 2048: 23.5, 23.7 and 26.5 ms), and the
// large one is not built.
int choose_tile(int64_t np, int64_t nq, int64_t steps, bool cut, bool bf16) {
    int best = 1;
    double least = 0.0;
    for (int shape = bf16 ? 0 : 1; shape < 3; ++shape) {
        const TileShape t = kTiles[shape];
        const int64_t tiles = ceil_div(np, t.p) * ceil_div(nq, t.q), rest = tiles % t.at_once;
        const int64_t part = bf16 ? kPartCost16 : kPartCost32;
        double last = rest > 0 ? (double)(steps + part) : 0.0;
        if (cut && rest > 0)
            for (int wanted = 2; wanted <= kMaxParts; ++wanted) {
                const HeadParts h = head_parts((int)steps, wanted);
                const int64_t k = h.parts;
                if (steps < kMinPart * k || rest * k > kMaxSlots) continue;
                const double c = (double)(ceil_div(rest * k, t.at_once) * (h.per + part) + k / 8)
                                 + (double)(rest * k) / ((bf16 ? 1 : 4) * t.join);
                if (c < last) last = c;
            }
        const double unit = shape == 0 ? 1.0 : shape == 1 ? (bf16 ? 0.62 : 0.5) : nq <= 32 ? 0.25 : bf16 ? 0.6 : 0.28;
        const double cost = unit * ((double)(tiles / t.at_once * (steps + part)) + last);
        if (least == 0.0 || cost < least) least = cost, best = shape;
    }
    return best;
}

// Few rows: the table is read once, whatever the tile, and what counts is how much of
// it is under way. One tile to a compute unit, all rows wide, with three or four
// stages in LDS instead of two, reads 32000 x 5120 bf16 for one row in 75 us (call;
// the other tiles 96), for 128 in 88 (105), for 192 in 98 (117), for 256 in 115 (130).
// A table of fewer tiles leaves compute units without one, which costs from about two
// rows a tile on (16000 x 4096: 160 rows 67 for 73, 256 rows 80 for 75). A table of more
// goes by the other tiles: 4096 wide, one row and 128 rows of 32768 entries take 78 and
// 81 us, of 33024 85 and 104, of 50257 114 and 120 (3.6 and 3.4 TB/s), of 128256 234 and
// 264 (4.5 and 4.0). fp32 is bound by its multiplying (1 row of 32000 x 4096 146 for 149, 48 rows 192 for 179).
int logits_tile(int64_t vocab, int64_t rows, int64_t steps, bool bf16) {
    const int64_t tiles = ceil_div(vocab, 128);
    if (bf16 && tiles <= 256 && rows <= 2 * tiles)
        for (int shape = 3; shape < 8; ++shape)
            if (rows <= kTiles[shape].q) return shape;
    return choose_tile(vocab, rows, steps, false, bf16);
}

// What one workgroup does in about a launch's time, 2.5 us on the device and more on
// the host, does not get one: rows and numbers of them that it sets to zero (1024 rows
// of 1000 x 64: 53.5 us so, 48.8 with a launch), and rounds in which each of its
// threads goes through 16 bytes, or each of its waves (each quarter of one, if there
// are few) through a row's statistics. e's turning into G also writes zeros, up to 64
// rows; those are quicker: three times as many rounds with them. With both gradients,
// 64 wide, bf16: 8 rows of 256 take 21.6 us for 23.4 with a launch, 32 of 500 (2
// rounds, 4 with the zeros) 26.4 for 27.8; 64 of 500 (4 and 4) 32.8 for 28.4, 16 of
// 1000 (2 and 8) 32.6 for 31.5, 1 of 16000 (2 and 125) 55.9 for 34.8; fp32: 4 of 300
// (0.4 and 6) 28.6 for 29.7, 8 of 500 (1 and 8) 32.1 either way.
constexpr int64_t kSmallRows = 256, kSmallZeros = 65536, kSmallRounds = 2;

void plan_small(const HeadArgs &a, HeadPlan &p) {
    const int64_t round = 1024 * (a.bf16 ? 8 : 4), rows = round_up(a.count, 64);
    const int64_t statistics = p.subtiles <= kFewStats ? ceil_div(a.count, 64) : ceil_div(a.count, 16) * ceil_div(p.subtiles, 512);
    p.idle_with_rows = a.grad_hidden && a.count <= kSmallRows && a.count * a.width <= kSmallZeros;
    p.pack_with_rows = p.pieces == 1 && rows * p.width_p <= kSmallRounds * round;
    p.softmax_with_loss = p.pieces == 1 && statistics <= kSmallRounds;
    p.turn_with_loss = p.softmax_with_loss && (a.grad_hidden || a.grad_table) && a.count * p.vocab_p <= kSmallRounds * round &&
                       rows * p.vocab_p <= 3 * kSmallRounds * round;
}

}  // namespace

HeadPlan plan_head(const HeadArgs &a, int64_t rows) {
    HeadPlan p = {};
    const int64_t es = a.bf16 ? 2 : 4, step = 128 / es;
    p.width_p = round_up(a.width, step);
    p.vocab_p = round_up(a.vocab, 128);
    p.pack_table = (uintptr_t)a.table % 16 || p.width_p != a.width;
    // a piece's e takes a GiB at most
    int64_t piece = rows > 0 ? rows : ((int64_t)1 << 30) / (p.vocab_p * es) / 256 * 256;
    if (rows <= 0) piece = piece < 256 ? 256 : piece > 262144 ? 262144 : piece;
    if (piece > a.count) piece = a.count;
    if (piece < 1) piece = 1;
    p.piece = piece;
    p.pieces = a.count > 0 ? ceil_div(a.count, piece) : (a.grad_table ? 1 : 0);
    p.piece_p = round_up(piece, 64);
    p.tile_logits = logits_tile(a.vocab, piece, p.width_p / step, a.bf16);
    p.sub = kTiles[p.tile_logits].sub;
    p.subtiles = round_up(a.vocab, kTiles[p.tile_logits].p) / p.sub;
    p.tile_hidden = choose_tile(a.width, piece, ceil_div(a.vocab, step), true, a.bf16);
    p.tile_table = choose_tile(a.width, a.vocab, ceil_div(piece, step), true, a.bf16);
    // parts of tiles that do not fill a round
    auto slots = [&](int shape, int64_t np, int64_t nq, int64_t steps) -> int {
        const TileShape t = kTiles[shape];
        const int64_t tiles = ceil_div(np, t.p) * ceil_div(nq, t.q);
        if (steps < 2 * kMinPart) return 0;
        const int64_t n = kMaxParts * (tiles < t.at_once ? tiles : t.at_once);
        return (int)(n < kMaxSlots ? n : kMaxSlots);
    };
    p.slots_hidden = a.grad_hidden ? slots(p.tile_hidden, a.width, piece, ceil_div(a.vocab, step)) : 0;
    p.slots_table = a.grad_table ? slots(p.tile_table, a.width, a.vocab, ceil_div(piece, step)) : 0;
    auto room = [](int slots, int shape) { return (int64_t)slots * kTiles[shape].p * kTiles[shape].q * 4; };
    const int64_t parts_h = room(p.slots_hidden, p.tile_hidden), parts_t = room(p.slots_table, p.tile_table);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += round_up(bytes, 256);
        return here;
    };
    const bool grads = a.grad_hidden || a.grad_table;
    p.sum_off = take(sizeof(HeadSums));
    p.map_off = take(8 * a.count);           // and their targets
    p.loss_off = a.losses ? -1 : take(4 * a.count);
    p.row_off = take(sizeof(HeadRow) * piece);
    p.stat_off = take(8 * piece * p.subtiles);
    p.hidden_off = take(p.piece_p * p.width_p * es);
    p.table_off = p.pack_table ? take(a.vocab * p.width_p * es) : -1;
    p.e_off = grads ? take(p.piece_p * p.vocab_p * es) : -1;
    p.gw_off = a.grad_table && a.table_grad_bf16 && p.pieces > 1 ? take(4 * a.vocab * a.width) : -1;
    p.parts_off = take(parts_h > parts_t ? parts_h : parts_t);
    p.bytes = at;
    plan_small(a, p);
    return p;
}

}  // namespace zk

extern "C" {

int zero_embed(const void *ids, int32_t id_bytes, int64_t count, const void *table, int64_t rows, int64_t width,
               zero_dtype dtype, double scale, const void *position_ids, const void *position_table,
               int64_t position_rows, const zero_drop *drop, void *out, zero_dtype out_dtype, hipStream_t stream) {
    CaptureScope scope(stream);
    zk::EmbedArgs a = {};
    int rc = check_table(rows, width, "table");
    if (rc) return rc;
    if (!valid_dtype(dtype) || !valid_dtype(out_dtype)) return fail(ZERO_EINVAL, "unknown dtype");
    if ((rc = check_count(count, width))) return rc;
    if ((rc = check_scale(scale))) return rc;
    if ((rc = check_drop(drop, &a.drop))) return rc;
    if ((rc = check_ids(ids, id_bytes, count, "ids"))) return rc;
    if ((rc = check_buffer(table, rows * width, dtype_size(dtype), "table"))) return rc;
    // no ids have no address: a call without rows may come with the table alone
    if (!position_ids != !position_table && (position_ids || count > 0))
        return fail(ZERO_EINVAL, "position ids and a position table come together");
    if (position_table) {
        if ((rc = check_table(position_rows, width, "position table"))) return rc;
        if ((rc = check_ids(position_ids, id_bytes, count, "position ids"))) return rc;
        if ((rc = check_buffer(position_table, position_rows * width, dtype_size(dtype), "position table"))) return rc;
    }
    if ((rc = check_buffer(out, count * width, dtype_size(out_dtype), "out"))) return rc;
    const int64_t bytes = count * width * dtype_size(out_dtype);
    if (overlap(out, bytes, table, rows * width * dtype_size(dtype)) || overlap(out, bytes, ids, count * id_bytes) ||
        overlap(out, bytes, position_table, position_rows * width * dtype_size(dtype)) ||
        overlap(out, bytes, position_ids, count * id_bytes) || holds_counter(out, bytes, drop))
        return fail(ZERO_EINVAL, "out overlaps an input");
    a.ids = ids;
    a.pos_ids = position_ids;
    a.wide_ids = id_bytes == 8;
    a.count = count;
    a.rows = rows;
    a.pos_rows = position_rows;
    a.width = width;
    a.table = table;
    a.pos_table = position_table;
    a.table_bf16 = dtype == ZERO_BF16;
    a.out_bf16 = out_dtype == ZERO_BF16;
    a.scale = (float)scale;
    a.out = out;
    const hipError_t e = zk::launch_embed(a, stream);
    return e == hipSuccess ? ZERO_OK : hip_fail(e, "zero_embed");
}

int zero_embed_grad_workspace(int64_t count, int64_t rows, int64_t width, int64_t *bytes) {
    int rc = check_table(rows, width, "table");
    if (rc) return rc;
    if ((rc = check_count(count, width))) return rc;
    if (!bytes) return fail(ZERO_EINVAL, "null bytes");
    const zk::EmbedGradPlan p = zk::plan_embed_grad(count, rows, width);
    if ((rc = check_sort(p, count, rows))) return rc;
    *bytes = p.bytes;
    return ZERO_OK;
}

int zero_embed_grad(const void *grad_out, zero_dtype grad_dtype, const void *ids, int32_t id_bytes, int64_t count,
                    int64_t rows, int64_t width, double scale, const zero_drop *drop, void *grad_table,
                    zero_dtype table_dtype, int32_t accumulate, void *workspace, int64_t workspace_bytes,
                    hipStream_t stream) {
    CaptureScope scope(stream);
    zk::EmbedGradArgs a = {};
    int rc = check_table(rows, width, "table");
    if (rc) return rc;
    if (!valid_dtype(grad_dtype) || !valid_dtype(table_dtype)) return fail(ZERO_EINVAL, "unknown dtype");
    if ((rc = check_count(count, width))) return rc;
    const zk::EmbedGradPlan p = zk::plan_embed_grad(count, rows, width);
    if ((rc = check_sort(p, count, rows))) return rc;
    if ((rc = check_scale(scale))) return rc;
    if ((rc = check_drop(drop, &a.drop))) return rc;
    if ((rc = check_ids(ids, id_bytes, count, "ids"))) return rc;
    if ((rc = check_buffer(grad_out, count * width, dtype_size(grad_dtype), "grad_out"))) return rc;
    if ((rc = check_buffer(grad_table, rows * width, dtype_size(table_dtype), "grad_table"))) return rc;
    const int64_t bytes = rows * width * dtype_size(table_dtype);
    if (overlap(grad_table, bytes, grad_out, count * width * dtype_size(grad_dtype)) ||
        overlap(grad_table, bytes, ids, count * id_bytes) || holds_counter(grad_table, bytes, drop))
        return fail(ZERO_EINVAL, "grad_table overlaps an input");
    if ((rc = check_workspace(workspace, workspace_bytes, p.bytes))) return rc;
    if (overlap(workspace, p.bytes, grad_out, count * width * dtype_size(grad_dtype)) ||
        overlap(workspace, p.bytes, grad_table, bytes) || overlap(workspace, p.bytes, ids, count * id_bytes) ||
        holds_counter(workspace, p.bytes, drop))
        return fail(ZERO_EINVAL, "workspace overlaps another buffer");
    a.grad_out = grad_out;
    a.grad_bf16 = grad_dtype == ZERO_BF16;
    a.ids = ids;
    a.wide_ids = id_bytes == 8;
    a.count = count;
    a.rows = rows;
    a.width = width;
    a.scale = (float)scale;
    a.out = grad_table;
    a.out_bf16 = table_dtype == ZERO_BF16;
    a.accumulate = accumulate != 0;
    a.workspace = static_cast<char *>(workspace);
    const hipError_t e = zk::launch_embed_grad(a, p, stream);
    return e == hipSuccess ? ZERO_OK : hip_fail(e, "zero_embed_grad");
}

int zero_dropout(const void *x, const void *add, void *out, int64_t count, zero_dtype dtype, const zero_drop *drop,
                 hipStream_t stream) {
    CaptureScope scope(stream);
    zk::DropoutArgs a = {};
    if (!valid_dtype(dtype)) return fail(ZERO_EINVAL, "unknown dtype %d", (int)dtype);
    if (count < 0) return fail(ZERO_EINVAL, "count must be >= 0 (got %lld)", (long long)count);
    if (ceil_div(count, 4) > kMaxUnits)
        return fail(ZERO_EUNSUPPORTED, "%lld elements are more than one call takes", (long long)count);
    if (!drop) return fail(ZERO_EINVAL, "drop is null");
    int rc = check_drop(drop, &a.drop);
    if (rc) return rc;
    const int64_t es = dtype_size(dtype);
    if ((rc = check_buffer(x, count, es, "x"))) return rc;
    if (add && (rc = check_buffer(add, count, es, "add"))) return rc;
    if ((rc = check_buffer(out, count, es, "out"))) return rc;
    // in place is element by element, a shifted overlap is not
    if ((out != x && overlap(out, count * es, x, count * es)) ||
        (add && out != add && overlap(out, count * es, add, count * es)))
        return fail(ZERO_EINVAL, "out overlaps an input without being it");
    if (holds_counter(out, count * es, drop)) return fail(ZERO_EINVAL, "out overlaps the dropout counter");
    a.x = x;
    a.add = add;
    a.out = out;
    a.bf16 = dtype == ZERO_BF16;
    a.count = count;
    const hipError_t e = zk::launch_dropout(a, stream);
    return e == hipSuccess ? ZERO_OK : hip_fail(e, "zero_dropout");
}

int zero_head_loss_workspace(int64_t count, int64_t vocab, int64_t width, zero_dtype dtype, int32_t grad_hidden,
                             int32_t grad_table, zero_dtype table_grad_dtype, int64_t piece_rows, int64_t *bytes) {
    int rc = head_sizes(count, vocab, width, dtype, piece_rows);
    if (rc) return rc;
    if (!valid_dtype(table_grad_dtype)) return fail(ZERO_EINVAL, "unknown dtype %d", (int)table_grad_dtype);
    if (!bytes) return fail(ZERO_EINVAL, "null bytes");
    zk::HeadArgs a = {};
    a.table = reinterpret_cast<const void *>(1);      // any alignment
    a.bf16 = dtype == ZERO_BF16;
    a.count = count;
    a.width = width;
    a.vocab = vocab;
    a.grad_hidden = grad_hidden ? bytes : nullptr;
    a.grad_table = grad_table ? bytes : nullptr;
    a.table_grad_bf16 = table_grad_dtype == ZERO_BF16;
    *bytes = zk::plan_head(a, piece_rows).bytes;
    return ZERO_OK;
}

int zero_head_loss(const void *hidden, const void *table, zero_dtype dtype, const void *targets, int32_t id_bytes,
                   int64_t count, int64_t vocab, int64_t width, const float *weights, int32_t mean, double grad_scale,
                   float *loss, float *losses, void *grad_hidden, void *grad_table, zero_dtype table_grad_dtype,
                   int32_t accumulate, int64_t piece_rows, void *workspace, int64_t workspace_bytes,
                   hipStream_t stream) {
    CaptureScope scope(stream);
    int rc = head_sizes(count, vocab, width, dtype, piece_rows);
    if (rc) return rc;
    if (!valid_dtype(table_grad_dtype)) return fail(ZERO_EINVAL, "unknown dtype %d", (int)table_grad_dtype);
    if (!std::isfinite((float)grad_scale))
        return fail(ZERO_EINVAL, "grad_scale must be finite in fp32 (got %g)", grad_scale);
    const int64_t es = dtype_size(dtype), gs = dtype_size(table_grad_dtype);
    if ((rc = check_ids(targets, id_bytes, count, "targets"))) return rc;
    if ((rc = check_buffer(hidden, count * width, es, "hidden"))) return rc;
    if ((rc = check_buffer(table, vocab * width, es, "table"))) return rc;
    if (weights && (rc = check_buffer(weights, count, 4, "weights"))) return rc;
    if ((rc = check_buffer(loss, 1, 4, "loss"))) return rc;
    if (losses && (rc = check_buffer(losses, count, 4, "losses"))) return rc;
    if (grad_hidden && (rc = check_buffer(grad_hidden, count * width, es, "grad_hidden"))) return rc;
    if (grad_table && (rc = check_buffer(grad_table, vocab * width, gs, "grad_table"))) return rc;
    zk::HeadArgs a = {};
    a.hidden = hidden;
    a.table = table;
    a.bf16 = dtype == ZERO_BF16;
    a.targets = targets;
    a.wide_ids = id_bytes == 8;
    a.count = count;
    a.width = width;
    a.vocab = vocab;
    a.weights = weights;
    a.mean = mean != 0;
    a.grad_scale = (float)grad_scale;
    a.loss = loss;
    a.losses = losses;
    a.grad_hidden = grad_hidden;
    a.grad_table = grad_table;
    a.table_grad_bf16 = table_grad_dtype == ZERO_BF16;
    a.accumulate = accumulate != 0;
    a.workspace = static_cast<char *>(workspace);
    const zk::HeadPlan p = zk::plan_head(a, piece_rows);
    if ((rc = check_workspace(workspace, workspace_bytes, p.bytes))) return rc;
    // every output and the workspace apart from everything else
    const struct {
        const void *p;
        int64_t bytes;
        bool written;
    } all[] = {{loss, 4, true},
               {losses, 4 * count, true},
               {grad_hidden, count * width * es, true},
               {grad_table, vocab * width * gs, true},
               {workspace, p.bytes, true},
               {hidden, count * width * es, false},
               {table, vocab * width * es, false},
               {targets, count * id_bytes, false},
               {weights, 4 * count, false}};
    for (const auto &x : all)
        for (const auto &y : all)
            if (&x != &y && x.written && overlap(x.p, x.bytes, y.p, y.bytes))
                return fail(ZERO_EINVAL, "an output or the workspace overlaps another buffer");
    const hipError_t e = zk::launch_head(a, p, stream);
    return e == hipSuccess ? ZERO_OK : hip_fail(e, "zero_head_loss");
}

}  // extern "C"
