// Internal interface between the host API of the vocabulary operators
// (vocab_api.hip) and their gfx950 kernels (vocab_kernels.hip,
// head_kernels.hip). Callers use include/zero.h.
#pragma once

#include "zero_internal.h"

namespace zk {

// Host checks that zero_api.hip implements (they set the thread's last error).
int fail(int code, const char *fmt, ...);
int hip_fail(hipError_t e, const char *what);
int check_range(const void *p, int64_t nbytes, const char *what);
// Skips check_range while `stream` is captured, for the scope's life.
class CaptureScope {
  public:
    explicit CaptureScope(hipStream_t stream);
    ~CaptureScope();
    CaptureScope(const CaptureScope &) = delete;
    CaptureScope &operator=(const CaptureScope &) = delete;
    bool capturing() const;

  private:
    bool prev_;
};

// Dropout: an element is kept where its 16 random bits are >= limit, and then
// multiplied by scale. limit == 0 means none.
struct Drop {
    uint32_t key0, key1;
    uint32_t limit;               // 0..65536
    float scale;
    uint64_t offset;
    const uint64_t *counter;      // device, added to offset; or null
};

struct EmbedArgs {
    const void *ids, *pos_ids;    // pos_ids null: no position table
    bool wide_ids;                // 64-bit ids
    int64_t count, rows, pos_rows, width;
    const void *table, *pos_table;
    bool table_bf16, out_bf16;
    float scale;
    Drop drop;
    void *out;
};
hipError_t launch_embed(const EmbedArgs &a, hipStream_t stream);

// One sorted token: its id, its row of grad_out, and the run of equal ids it
// is in, as [begin, end) of the sorted list.
struct SortedToken {
    int32_t id, row, begin, end;
};
// Ids are spread over the sorting workgroups by their remainder, at most
// kSortIds to each.
constexpr int kSortIds = 512;
constexpr int kSortWaves = 16;
struct EmbedGradPlan {
    int sort_groups_log2;         // workgroups of the sort
    int ids_per_group;
    int span;                     // sorted tokens one wave adds up; 1: a run
    int64_t spans;
    int64_t sorted_off, count_off, partial_off, bytes;   // workspace layout
};
// Up to so many tokens the sums go by runs: 128 tokens of 768 columns take 8.1 us for
// 12.5 by spans, 9.8 for 11.4 if they are one id; 256 take 8.4 for 12.8, and 13.2 for 12.
constexpr int kRunTokens = 256;
// Columns of one wave in the sums.
constexpr int kSpanCols = 512;
EmbedGradPlan plan_embed_grad(int64_t count, int64_t rows, int64_t width);
struct EmbedGradArgs {
    const void *grad_out;
    bool grad_bf16;
    const void *ids;
    bool wide_ids;
    int64_t count, rows, width;
    float scale;
    Drop drop;
    void *out;
    bool out_bf16, accumulate;
    char *workspace;
};
hipError_t launch_embed_grad(const EmbedGradArgs &a, const EmbedGradPlan &p, hipStream_t stream);

struct DropoutArgs {
    const void *x, *add;          // add null: none
    void *out;
    bool bf16;
    int64_t count;
    Drop drop;
};
hipError_t launch_dropout(const DropoutArgs &a, hipStream_t stream);

// ---- softmax cross entropy against a table (head_kernels.hip)
// What the call finds out first: how many rows take part, their weights' sum
// and the largest, and what both gradients are multiplied by.
struct HeadSums {
    double weight;
    int64_t rows;
    float most;                   // largest |weight|
    float scale;                  // grad_scale * most (/ the weights' sum)
};
// A row of at most so many statistics is a quarter wave's in the loss's workgroup.
constexpr int kFewStats = 64;
// Of each row that takes part, in the order of the piece.
struct HeadRow {
    float top;                    // largest z * log2(e)
    float inv;                    // share / sum of exponentials
    float share;                  // weight / most
    float target;                 // z_y * log2(e)
};
// Tiles of the products: rows of P and of Q, rows of P to a wave, and workgroups
// that run at a time: one, two or three on each of 256 compute units, as LDS lets
// them.
struct TileShape {
    int p, q, sub, at_once;
    int join;                     // parts that are joined in the time of a stage
};
constexpr TileShape kTiles[] = {{256, 256, 128, 256, 11}, {128, 128, 64, 512, 25}, {128, 32, 32, 768, 55},
                                // for the logits of few rows (logits_tile), not cut
                                {128, 32, 32, 256, 1}, {128, 64, 32, 256, 1}, {128, 128, 64, 256, 1},
                                {128, 192, 64, 256, 1}, {128, 256, 64, 256, 1}};
// A part of a tile: at most kMaxParts of at least kMinPart stages. What it takes
// besides, in stages, which take several times as long with fp32, where also that
// many more parts are joined in a stage's time.
constexpr int kMaxParts = 64, kMinPart = 8, kPartCost16 = 8, kPartCost32 = 2;
// Stages of each of about k parts of `steps` stages, the last one's the rest, and
// how many parts that makes: none is without a stage.
struct HeadParts {
    int per, parts;
};
__host__ __device__ inline HeadParts head_parts(int steps, int k) {
    const int per = (steps + k - 1) / k;
    return {per, per > 0 ? (steps + per - 1) / per : 1};
}
struct HeadPlan {
    int64_t piece, pieces;        // rows of hidden in a piece
    int64_t width_p, vocab_p, piece_p;   // extents padded for the products' long axes
    bool pack_table;              // table copied to aligned, padded rows
    int tile_logits, tile_hidden, tile_table;   // shapes of the three products' tiles
    int sub;                      // vocabulary entries that share a statistic
    int64_t subtiles;             // statistics of a row
    int slots_hidden, slots_table;       // room for parts of the gradients' tiles
    // small calls: what a kernel of one workgroup does besides, instead of a launch
    bool idle_with_rows, pack_with_rows, softmax_with_loss, turn_with_loss;
    // workspace offsets in bytes; -1: not there
    int64_t sum_off, map_off, loss_off, row_off, stat_off, hidden_off, table_off, e_off, gw_off,
        parts_off, bytes;
};
struct HeadArgs {
    const void *hidden, *table;
    bool bf16;
    const void *targets;
    bool wide_ids;
    int64_t count, width, vocab;
    const float *weights;
    bool mean;
    float grad_scale;
    float *loss, *losses;
    void *grad_hidden, *grad_table;
    bool table_grad_bf16, accumulate;
    char *workspace;
};
// rows: the most rows of hidden in one piece (0: by the memory of a piece).
HeadPlan plan_head(const HeadArgs &a, int64_t rows);
hipError_t launch_head(const HeadArgs &a, const HeadPlan &p, hipStream_t stream);

}  // namespace zk
