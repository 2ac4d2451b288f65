// Softmax cross entropy of hidden states against a vocabulary table, with the
// gradients of both, for gfx950.
//
//   z_iv = h_i . W_v,  l_i = log sum_v exp(z_iv) - z_iy
//   G_iv = w_i (exp(z_iv) / sum_u exp(z_iu) - [v = y]),  dh_i = s sum_v G_iv W_v,
//   dW_v = s sum_i G_iv h_i
//
// Three products on the matrix cores, tile by tile through LDS: the logits of rows
// with rows (both operands contiguous along the long axis), the gradients with one
// operand, or both, across it. The first one's epilogue takes each tile's maximum
// and sum of exponentials per row, in binary32 from the accumulators, and leaves
// e = exp(z - its tile's maximum) instead of z: e needs 2 bytes where z would need 4
// for the same p, for e's relative error is p's. With the row's maximum and sum
// known, one pass turns e into G, the operand of the other two products. w are the
// weights over the largest, and s the rest of the gradient's scale, which multiplies
// the products' binary32 sums: rounded to bf16 with s inside, the -s of the many
// entries with p = 0 would all be off by the same; so they are -1 and exact. Rows
// that take no part (target outside the table, weight 0) are left out of all products.
//
// Bound by the products, under which the clock falls from 2400 MHz to 2150 or 2220:
// GPT-2's head (8192 rows of 768 against 50257) takes 2.10 ms with both gradients,
// three products of 650, 559 and 556 us (970 to 1140 TFLOP/s; library products of
// these shapes, at 1990 to 2080 MHz, 574, 637 and 666) and 270 for e's turning into G;
// 6553 rows of 4096 against 32000 take 4.5 to 4.6 ms, three of 1389, 1427 and 1465
// (1170 to 1240 TFLOP/s; the library's 1171, 1751 and 1578). With fp32 1023 x 16001 x
// 1025 takes 0.96 ms, three of 282 to 312 us (108 to 119 TFLOP/s; a library product
// of 8192^3 153).
#include "vocab_internal.h"

namespace zk {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((address_space(3))) void lds_void;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr double kLn2 = 0.693147180559945309417;
// e of bf16 operands is held in fp16 as e * 2^15: 11 bits for e >= 2^-29, and
// what is below 2^-40 of its tile's largest becomes zero.
constexpr float kScaleLog2 = 15.0f;

__host__ __device__ constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
__host__ __device__ constexpr int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// To bf16, nearest, ties to even, NaN kept: two to an instruction.
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    typedef __attribute__((ext_vector_type(2))) float f32x2_t;
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
    const f32x2_t x = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2_t));
}
__device__ __forceinline__ float widen(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

template <bool BF16> struct Elem { using type = float; };
template <> struct Elem<true> { using type = uint16_t; };

__device__ __forceinline__ int64_t load_id(const void *ids, bool wide, int64_t i) {
    return wide ? static_cast<const int64_t *>(ids)[i] : (int64_t) static_cast<const int32_t *>(ids)[i];
}

// Whether row i has a loss.
__device__ __forceinline__ bool takes_part(const HeadArgs &a, int64_t i) {
    return (uint64_t)load_id(a.targets, a.wide_ids, i) < (uint64_t)a.vocab && !(a.weights && a.weights[i] == 0.0f);
}

__device__ __forceinline__ int piece_rows(const HeadSums *s, int64_t first, int64_t piece) {
    const int64_t n = s->rows - first;
    return __builtin_amdgcn_readfirstlane((int)(n < 0 ? 0 : n < piece ? n : piece));
}

// ------------------------------------------------------- copies
// Numbers c.. of `dst`, 16 bytes on a 16-byte address, = those of `src`, cols
// numbers anywhere, and zeros behind them; all zeros for a null src.
template <bool BF16>
__device__ __forceinline__ void pack_chunk(const void *src, int64_t cols, void *dst, int64_t c) {
    using T = typename Elem<BF16>::type;
    const T *s = static_cast<const T *>(src);
    constexpr int V = 16 / sizeof(T);
    T x[V];
    if (s && c + V <= cols) {
        __builtin_memcpy(x, s + c, sizeof x);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) x[k] = s && c + k < cols ? s[c + k] : (T)0;
    }
    __builtin_memcpy(__builtin_assume_aligned(static_cast<T *>(dst) + c, 16), x, sizeof x);
}

// Chunk c of row r of the packed hidden states of a piece with n rows.
template <bool BF16>
__device__ __forceinline__ void pack_hidden(const HeadArgs &a, const int32_t *map, int64_t first, int n, int64_t r, int64_t c,
                                            void *packed, int64_t width_p) {
    constexpr int es = BF16 ? 2 : 4;
    const char *src = r < n ? static_cast<const char *>(a.hidden) + (int64_t)map[first + r] * a.width * es : nullptr;
    pack_chunk<BF16>(src, a.width, static_cast<char *>(packed) + r * width_p * es, c);
}

// The rows of a piece, and zeros up to a whole stage. A workgroup to a row.
template <bool BF16>
__global__ void __launch_bounds__(256)
pack_hidden_kernel(HeadArgs a, const int32_t *map, const HeadSums *sums, int64_t first, int64_t piece, void *packed, int64_t width_p) {
    constexpr int V = BF16 ? 8 : 4;
    const int n = piece_rows(sums, first, piece);
    if (blockIdx.x < round_up(n, 64))
        for (int64_t c = threadIdx.x * V; c < width_p; c += 256 * V)
            pack_hidden<BF16>(a, map, first, n, blockIdx.x, c, packed, width_p);
}

// A table whose rows are not whole stages on 16-byte addresses.
template <bool BF16>
__global__ void __launch_bounds__(256) pack_table_kernel(HeadArgs a, void *packed, int64_t width_p) {
    constexpr int es = BF16 ? 2 : 4, V = 16 / es;
    const int64_t r = blockIdx.x;
    for (int64_t c = threadIdx.x * V; c < width_p; c += 256 * V)
        pack_chunk<BF16>(static_cast<const char *>(a.table) + r * a.width * es, a.width, static_cast<char *>(packed) + r * width_p * es, c);
}

// ------------------------------------------------------- which rows
// A wave: the gradient of row i, which takes no part, is zero.
__device__ __forceinline__ void idle_row(const HeadArgs &a, int64_t i, int lane) {
    for (int64_t c = lane; c < a.width; c += 64)
        if (a.bf16) static_cast<uint16_t *>(a.grad_hidden)[i * a.width + c] = 0;
        else static_cast<float *>(a.grad_hidden)[i * a.width + c] = 0.0f;
}

// One workgroup: the rows that take part, in order, with their targets, and their
// weights' sum; the others' losses, zeros. In small calls also the others'
// gradients (idle), and the rows packed. A wave takes kRows * 64 rows at a time,
// all asked for before the first is used.
template <bool BF16, int kRows>
__global__ void __launch_bounds__(1024)
rows_kernel(HeadArgs a, HeadSums *sums, int32_t *map, int32_t *target, float *losses, bool idle, void *packed, int64_t width_p) {
    __shared__ int32_t found[16];
    __shared__ uint64_t on[16];
    __shared__ double parts[16];
    __shared__ float tops[16];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    int64_t base = 0;
    double weight = 0.0;
    float most = 0.0f;
    for (int64_t i0 = 0; i0 < a.count; i0 += 1024 * kRows) {
        const int64_t first = i0 + 64 * kRows * wave + lane;
        int64_t y[kRows];
        float w[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t i = first + 64 * k;
            y[k] = i < a.count ? load_id(a.targets, a.wide_ids, i) : -1;
            w[k] = !a.weights ? 1.0f : i < a.count ? a.weights[i] : 0.0f;
        }
        uint64_t mask[kRows];
        int mine = 0;
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const bool part = (uint64_t)y[k] < (uint64_t)a.vocab && w[k] != 0.0f;   // as takes_part()
            mask[k] = __ballot(part);
            mine += __popcll(mask[k]);
            if (part) {
                weight += (double)w[k];
                most = fmaxf(most, fabsf(w[k]));
            }
        }
        if (lane == 0) found[wave] = mine, on[wave] = mask[0];
        __syncthreads();
        if (idle)                                 // one round, of one row a thread
            for (int i = wave; i < a.count; i += 16)
                if (!(on[i / 64] >> (i % 64) & 1)) idle_row(a, i, lane);
        int64_t at = base;
        for (int x = 0; x < 16; ++x) {
            if (x < wave) at += found[x];
            base += found[x];
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            if (mask[k] >> lane & 1) {
                const int64_t to = at + __popcll(mask[k] & ((1ull << lane) - 1));
                map[to] = (int32_t)(first + 64 * k);
                target[to] = (int32_t)y[k];
            }
            at += __popcll(mask[k]);
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t i = first + 64 * k;
            if (i < a.count && !(mask[k] >> lane & 1)) losses[i] = 0.0f;
        }
        __syncthreads();
    }
    for (int s = 32; s; s /= 2) {
        weight += __shfl_xor(weight, s);
        most = fmaxf(most, __shfl_xor(most, s));
    }
    if (lane == 0) parts[wave] = weight, tops[wave] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
        weight = 0.0;
        for (int w = 0; w < 16; ++w) {
            weight += parts[w];
            most = fmaxf(most, tops[w]);
        }
        if (!(most > 0.0f)) most = 1.0f;
        sums->weight = weight;
        sums->rows = base;
        sums->most = most;
        sums->scale = (float)((double)a.grad_scale * (double)most / (a.mean && weight != 0.0 ? weight : 1.0));
    }
    if (packed) {                                 // the map is this workgroup's own, and synchronised
        constexpr int V = BF16 ? 8 : 4;
        const uint32_t per_row = (uint32_t)(width_p / V);
        for (uint32_t k = threadIdx.x; k < (uint32_t)round_up(base, 64) * per_row; k += 1024)
            pack_hidden<BF16>(a, map, 0, (int)base, k / per_row, (int64_t)(k % per_row) * V, packed, width_p);
    }
}

// ------------------------------------------------------- the product
// out[q][p] = sum_k P[p][k] Q[q][k]; lines of P and Q are 16-byte aligned, and
// those along k a whole number of 128-byte stages. A workgroup makes BP x BQ outputs
// with WP x WQ waves; a stage of both operands, 128 bytes of k, goes straight from
// memory to LDS while the stage before it is multiplied. What is not kept, and why:
// the 32 x 32 x 16 instruction, fewer cycles but 5% more time (4.76 ms for 4.54);
// 128 x 128 outputs to a wave (registers spill).
//
// LDS holds a row's 128 bytes as eight 16-byte chunks, chunk c at place
// c ^ (row % 8): then the 16 rows that a fragment reads at one chunk lie on
// different banks. A load to LDS writes lane after lane, so the exchange is made
// in the addresses it reads from. An operand across k ([k][row]) is brought as it
// lies, and turned as it is read: by ds_read_b64_tr_b16, or number by number (fp32).

enum Epilogue { kLogits, kBf16, kF32 };

struct Product {
    const void *p, *q;
    int64_t ldp, ldq;             // bytes
    int64_t np, nq;               // rows
    int64_t kp, kq;               // lines of operands across the long axis
    int64_t steps;                // of 128 bytes on the long axis
    int slots;                    // room for parts of tiles (0: tiles are not cut)
    float *parts;
    // with sums: rows of the piece, which bound nq or the long axis
    const HeadSums *sums;
    int64_t first, piece;
    bool piece_is_q, piece_is_k;
    // kLogits
    const int32_t *target;        // of the rows of Q
    f32x2 *stat;
    HeadRow *row;
    int64_t subtiles;
    void *e;                      // null: not wanted
    int64_t lde;                  // elements
    // kBf16: out = scaled product + f32_in + old out; kF32: f32 = scaled product + f32_in
    const int32_t *map;           // rows of the output, if they are others
    float *f32;
    const float *f32_in;          // or null
    void *out;
    bool add_out;
    int64_t ldo;                  // elements, of f32, f32_in and out
};

// Which workgroup makes what. Tiles are dealt to `at_once` workgroups, as many as
// run at a time; those of a last, incomplete round are cut along the long axis
// into parts, whose sums go to slots and are joined by another kernel. 7B list's
// grad_hidden of 6553 rows: 416 tiles on 256 compute units, 160 of them in three
// parts, took 1.45 ms where two whole rounds took 1.68.
struct Schedule {
    int tiles_p, tiles_q, whole, cut, parts, units;
    int steps, per;               // of a whole tile, of a part
};

// Every lane has the same value; the compiler is not always aware of it.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

__device__ __forceinline__ Schedule schedule(const Product &g, int bp, int bq, int es, int at_once, int join, int part_cost) {
    Schedule s;
    int nq = (int)g.nq;
    s.steps = (int)g.steps;
    if (g.sums) {
        const int n = piece_rows(g.sums, g.first, g.piece);
        if (g.piece_is_q) nq = n;
        if (g.piece_is_k) s.steps = (n * es + 127) / 128;
    }
    s.tiles_p = ((int)g.np + bp - 1) / bp;
    s.tiles_q = (nq + bq - 1) / bq;
    const int tiles = s.tiles_p * s.tiles_q;
    s.cut = uniform(tiles % at_once);
    s.whole = tiles - s.cut;
    s.parts = 1;
    s.per = s.steps;
    if (s.cut > 0 && g.slots > 0) {
        // Lane k - 1 works out what about k parts would take, in steps: rounds of parts
        // with a part's own cost, the parts' traffic, and the joining one after the other.
        const int wanted = threadIdx.x % 64 + 1;
        const HeadParts h = head_parts(s.steps, wanted);
        const int k = h.parts;
        int cost = ((s.cut * k + at_once - 1) / at_once) * (h.per + part_cost) + (k > 1 ? s.cut * k / join + k / 8 : 0);
        if (k > 1 && (s.steps < kMinPart * k || s.cut * k > g.slots)) cost = 0x1FFFFFF;
        int best = (cost < 0x1FFFFFF ? cost : 0x1FFFFFF) * 64 + (wanted - 1);
        for (int d = 32; d; d /= 2) {
            const int other = __shfl_xor(best, d);
            best = other < best ? other : best;
        }
        const HeadParts chosen = head_parts(s.steps, best % 64 + 1);
        s.parts = uniform(chosen.parts);
        s.per = uniform(chosen.per);
    }
    s.units = s.whole + s.cut * s.parts;
    return s;
}

// The tile at place t of n: workgroups go round robin over the 8 XCDs, so each
// XCD gets a run of neighbouring tiles, in groups of 8 along p, to share its L2.
__device__ __forceinline__ void place(const Schedule &s, int t, int n, int first, int *p, int *q) {
    const int per = n / 8, rest = n % 8, x = t % 8;
    t = first + x * per + (x < rest ? x : rest) + t / 8;
    const int group = t / (8 * s.tiles_q), in = t % (8 * s.tiles_q);
    const int gp = s.tiles_p - 8 * group < 8 ? s.tiles_p - 8 * group : 8;
    *p = uniform(8 * group + in % gp);
    *q = uniform(in / gp);
}

struct Unit {
    int64_t p0, q0;
    int k0, steps, slot;          // slot < 0: a whole tile
};

__device__ __forceinline__ Unit unit_of(const Schedule &s, int u, int bp, int bq) {
    Unit r;
    int p, q;
    r.k0 = 0;
    r.steps = s.steps;
    r.slot = -1;
    if (u < s.whole || s.parts == 1) {
        if (u < s.whole) place(s, u, s.whole, 0, &p, &q);
        else place(s, u - s.whole, s.cut, s.whole, &p, &q);
    } else {
        const int part = uniform((u - s.whole) / s.cut), t = u - s.whole - part * s.cut;
        place(s, t, s.cut, s.whole, &p, &q);
        r.k0 = s.per * part;
        r.steps = s.steps - r.k0 < s.per ? s.steps - r.k0 : s.per;
        r.slot = t * s.parts + part;
    }
    r.p0 = (int64_t)p * bp;
    r.q0 = (int64_t)q * bq;
    return r;
}

template <bool BF16> struct Frag { using type = f32x4; };
template <> struct Frag<true> { using type = bf16x8; };

// 16 x 16 outputs from 16 bytes a lane: lanes 16g..16g+15 hold 16 rows' g-th
// chunk. binary32 takes four instructions, the k-th on every chunk's k-th number.
__device__ __forceinline__ f32x4 mma(bf16x8 p, bf16x8 q, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(p, q, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(f32x4 p, f32x4 q, f32x4 c) {
#pragma unroll
    for (int k = 0; k < 4; ++k) c = __builtin_amdgcn_mfma_f32_16x16x4f32(p[k], q[k], c, 0, 0, 0);
    return c;
}

// 16 bytes a lane, from base + from, to LDS at `lds` + 16 * lane; nothing from
// base + bytes on is read. In assembly, since the compiler would otherwise wait
// for all such loads before it reads LDS across lanes (ds_read_b64_tr_b16); the
// waits are the loop's own. No vector register is written; m0 is, which the compiler
// has to know of, though it warns of every reserved register that is named.
__device__ __forceinline__ void load_to_lds(const char *base, uint32_t bytes, int from, uint32_t lds) {
    typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
    const u32x4 r = {(uint32_t)(uintptr_t)base, (uint32_t)((uintptr_t)base >> 32) & 0xFFFFu, bytes, 0x00027000u};
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(from), "s"(r)
                 : "m0", "memory");
#pragma clang diagnostic pop
}

// One operand's tile of a stage: B rows and 128 bytes of the long axis, from
// rows along it ([row][k], T false) or across it ([k][row], T true).
template <bool BF16, bool T, int B, int LOADS>
struct Operand {
    static constexpr int kEs = BF16 ? 2 : 4, kSteps = 128 / kEs;
    static constexpr int kLine = T ? B * kEs : 128;           // bytes of a line in LDS
    int at[LOADS];                                            // what each load's lane reads
    int step;                                                 // bytes from stage to stage
    const char *base;                                         // of the next stage
    int64_t room;                                             // bytes from there to the operand's end

    // Where the 16-byte chunk at place c of line k comes from.
    static __device__ __forceinline__ int source(int k, int c) {
        if (!T) return c ^ (k % 8);
        if (BF16) return c ^ ((((k & 3) | ((k >> 1) & 4)) << 1) & (kLine / 16 - 1));
        return c ^ (((k >> 2) & 3) << 2 & (kLine / 16 - 1));
    }
    __device__ __forceinline__ void init(int wave, int lane, int ld) {
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            const int byte = (wave * LOADS + j) * 1024 + lane * 16, line = byte / kLine;
            at[j] = line * ld + source(line, byte % kLine / 16) * 16;
        }
        step = T ? kSteps * ld : 128;
    }
    // Rows behind the operand's last, and columns behind a line's (T), bring
    // whatever is there or nothing: they make outputs that are not stored.
    __device__ __forceinline__ void begin(const void *operand, int64_t first, int64_t ld, int64_t lines, int k0) {
        const int64_t off = (T ? first * kEs : first * ld) + (int64_t)k0 * step;
        base = static_cast<const char *>(operand) + off;
        room = lines * ld - off;
    }
    // lds: the operand's place in the stage. LAST (T): of a stage with fewer than
    // kSteps lines (`left` >= 1) those behind are read as the last; they meet zeros
    // of the other operand, and LDS might hold a NaN.
    template <bool LAST>
    __device__ __forceinline__ void load(uint32_t lds, int wave, int lane, int left, int ld) {
        const uint32_t bytes = room <= 0 ? 0u : room < 0xFFFFFFFFll ? (uint32_t)room : 0xFFFFFFFFu;
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            int from = at[j];
            if (LAST) {
                const int line = ((wave * LOADS + j) * 1024 + lane * 16) / kLine;
                if (line >= left) from -= (line - (left - 1)) * ld;
            }
            load_to_lds(base, bytes, from, lds + (wave * LOADS + j) * 1024);
        }
        base += step;
        room -= step;
    }
    // Fragment: 16 rows from row0 (a multiple of 16), half h of the stage.
    static __device__ __forceinline__ typename Frag<BF16>::type read(const char *lds, int row0, int h, int lane) {
        const int g = lane / 16, s = lane % 16;
        if constexpr (!T) {
            const int r = row0 + s;
            return *reinterpret_cast<const typename Frag<BF16>::type *>(lds + r * 128 + (((4 * h + g) ^ (lane % 8)) * 16));
        } else if constexpr (BF16) {
            // 16 lanes bring 4 lines of 16 numbers and get 4 lines' numbers of one row each
            typedef __attribute__((ext_vector_type(4))) short s16x4;
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            const int k = 32 * h + 8 * g + s / 4;
            const int c = row0 / 8 + s % 4 / 2;                // chunk of the four numbers
            const char *p = lds + k * kLine + source(k, c) * 16 + (s % 2) * 8;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * kLine));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            f32x4 v;
            const int k = 16 * h + 4 * g;
            const char *p = lds + k * kLine + source(k, row0 / 4 + s / 4) * 16 + (s % 4) * 4;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const float *>(p + e * kLine);
            return v;
        }
    }
};

template <bool BF16, int EPI, bool TP, bool TQ, int BP, int BQ, int WP, int WQ, int AT_ONCE, int JOIN, int DEPTH>
__device__ __forceinline__ void product(const Product &g) {
    constexpr int kWaves = WP * WQ;
    constexpr int kP = BP / WP, kQ = BQ / WQ;                 // outputs of a wave
    constexpr int kI = kP / 16, kJ = kQ / 16;                 // its fragments
    constexpr int kLoadsP = BP / 8 / kWaves, kLoadsQ = BQ / 8 / kWaves;
    static_assert(kLoadsP * 8 * kWaves == BP && kLoadsQ * 8 * kWaves == BQ, "whole loads");
    constexpr int kStage = (BP + BQ) * 128;
    using F = typename Frag<BF16>::type;
    using OpP = Operand<BF16, TP, BP, kLoadsP>;
    using OpQ = Operand<BF16, TQ, BQ, kLoadsQ>;
    // Outputs of two bytes are turned in LDS, 16 rows of q at a time, a wave its own.
    constexpr bool kTurned = EPI == kBf16 || (EPI == kLogits && BF16);
    constexpr int kTurn = kTurned ? 16 * kP * 2 : 0;
    __shared__ __align__(1024) char lds[DEPTH * kStage + kWaves * kTurn];

    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wp = wave / WQ, wq = wave % WQ;
    const Schedule sc = schedule(g, BP, BQ, OpP::kEs, AT_ONCE, JOIN, BF16 ? kPartCost16 : kPartCost32);
    const int64_t nq = g.sums && g.piece_is_q ? piece_rows(g.sums, g.first, g.piece) : g.nq;
    if ((int)blockIdx.x >= sc.units) return;

    // The loads run DEPTH stages ahead of the products, over the ends of units.
    OpP op;
    OpQ oq;
    op.init(wave, lane, (int)g.ldp);
    oq.init(wave, lane, (int)g.ldq);
    int lines = 0;                // of P left (TP: the table's rows are not padded)
    int next = blockIdx.x, left = 0, issued = 0;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void *)lds);
    auto begin = [&]() {
        const Unit u = unit_of(sc, next, BP, BQ);
        op.begin(g.p, u.p0, g.ldp, TP ? g.kp : g.np, u.k0);
        oq.begin(g.q, u.q0, g.ldq, TQ ? g.kq : nq, u.k0);
        if (TP) lines = (int)g.kp - u.k0 * OpP::kSteps;
        left = u.steps;
    };
    auto load = [&](int buf) {
        if (left == 0) return;
        const uint32_t s = lds0 + buf * kStage;
        if (TP && lines < OpP::kSteps) op.template load<true>(s, wave, lane, lines, (int)g.ldp);
        else op.template load<false>(s, wave, lane, 0, 0);
        oq.template load<false>(s + BP * 128, wave, lane, 0, 0);
        lines -= OpP::kSteps;
        if (DEPTH > 2) ++issued;
        if (--left == 0) {
            next += gridDim.x;
            if (next < sc.units) begin();
        }
        asm volatile("" : "+s"(left));            // one loop, not one for each way it can end
    };

    f32x4 acc[kI][kJ];
    // A stage is multiplied in four parts: part c takes half c / 2 of the long axis
    // and half c % 2 of the wave's rows of P.
    F fp[2][kI / 2], fq[2][kJ];
    auto read = [&](int buf, int c) {
        const char *s = lds + buf * kStage;
        if (c % 2 == 0)
#pragma unroll
            for (int j = 0; j < kJ; ++j) fq[c / 2][j] = OpQ::read(s + BP * 128, wq * kQ + 16 * j, c / 2, lane);
#pragma unroll
        for (int i = 0; i < kI / 2; ++i) fp[c % 2][i] = OpP::read(s, wp * kP + 16 * (c % 2 * (kI / 2) + i), c / 2, lane);
    };
    auto multiply = [&](int c) {
#pragma unroll
        for (int i = 0; i < kI / 2; ++i)
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                f32x4 &x = acc[c % 2 * (kI / 2) + i][j];
                x = mma(fp[c % 2][i], fq[c / 2][j], x);
            }
    };

    int target[kJ];
    auto targets = [&](int u) {
        if constexpr (EPI == kLogits) {
            if (u >= sc.units) return;
            const int64_t q = unit_of(sc, u, BP, BQ).q0 + wq * kQ + lane % 16;
#pragma unroll
            for (int j = 0; j < kJ; ++j) target[j] = q + 16 * j < nq ? g.target[g.first + q + 16 * j] : -1;
        }
    };
    // This wave's loads have arrived. The compiler does not count the loads to LDS;
    // it is told here, where nothing is left to wait for, that the targets are in.
    auto arrived = [&]() {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        if constexpr (EPI == kLogits)
#pragma unroll
            for (int j = 0; j < kJ; ++j) asm volatile("" : "+v"(target[j]));
    };

    if (sc.steps > 0) begin();
#pragma unroll
    for (int b = 0; b < DEPTH; ++b) load(b);
    targets(blockIdx.x);
    arrived();
    asm volatile("s_barrier" ::: "memory");
    read(0, 0);
    int stage = 0;
    for (int unit = blockIdx.x; unit < sc.units; unit += gridDim.x) {
        const Unit u = unit_of(sc, unit, BP, BQ);
#pragma unroll
        for (int i = 0; i < kI; ++i)
#pragma unroll
            for (int j = 0; j < kJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        // Each part is read while the one before is multiplied. When the last part of a
        // stage has been read by all, the loads of the stage after the next go to its
        // place, so a load has nearly a stage's time to arrive and a wave meets one
        // barrier a stage, with products still to do. A unit's first part is read with
        // the last of the unit before, and its first DEPTH stages have arrived before
        // that one's outputs are stored.
        for (int k = 0; k < u.steps; ++k) {
            const int buf = DEPTH == 2 ? (stage + k) & 1 : (unsigned)(stage + k) % DEPTH;
            int later = k;
            asm volatile("" : "+s"(later));       // no first round of its own
            read(buf, 1);
            __builtin_amdgcn_sched_barrier(0);    // the reads go first, whatever the scheduler thinks
            multiply(0);
            __builtin_amdgcn_sched_barrier(0);
            read(buf, 2);
            __builtin_amdgcn_sched_barrier(0);
            multiply(1);
            __builtin_amdgcn_sched_barrier(0);
            read(buf, 3);
            __builtin_amdgcn_sched_barrier(0);
            multiply(2);
            if (DEPTH == 2) {
                if (later > 0) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            } else {
                // all but the loads of the stages after the next: they arrive in order
                constexpr int kLoads = kLoadsP + kLoadsQ;
                const int after = uniform(issued - (stage + k) - 2);
                if (after >= 2) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kLoads) : "memory");
                else if (after == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads) : "memory");
                else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            }
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            load(buf);
            read(DEPTH == 2 ? buf ^ 1 : (unsigned)(buf + 1) % DEPTH, 0);    // after the last unit: of no use, but there
            __builtin_amdgcn_sched_barrier(0);
            multiply(3);
        }
        stage += u.steps;

        // A lane holds outputs p = pw + 16 i + r, r < 4, of q = qw + 16 j. What is
        // stored is stored after the loads under way have arrived: the wait for the
        // next stage would wait for the stores as well.
        const int64_t pw = u.p0 + wp * kP + lane / 16 * 4, qw = u.q0 + wq * kQ + lane % 16;
        const bool whole = u.p0 + BP <= g.np;
        char *turn = lds + DEPTH * kStage + wave * kTurn;
        // whole vectors: those go past the caches, parts of lines would be slow there
        const bool aligned = EPI == kLogits || (((uintptr_t)g.out | (uintptr_t)(2 * g.ldo)) % 16 == 0);
        // 16 rows of kP numbers of two bytes; 16-byte chunk c of row r at c ^ r.
        constexpr int kChunks = kP / 8;
        auto put = [&](int i, const uint16_t *h) {
            const int r = lane % 16, c = 2 * i + lane / 32;
            __builtin_memcpy(__builtin_assume_aligned(turn + r * kP * 2 + (c ^ (r % kChunks)) * 16 + lane / 16 % 2 * 8, 8), h, 8);
        };
        // Rows j of the turned numbers to `out`, whole lines of the wave's columns.
        auto send = [&](int j, uint16_t *out, int64_t ld, int64_t np) {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_wave_barrier();
            constexpr int kDown = 64 / kChunks;
            const int c = lane % kChunks;
            const int64_t p = u.p0 + wp * kP + c * 8;
#pragma unroll
            for (int r0 = 0; r0 < 16; r0 += kDown) {
                const int r = r0 + lane / kChunks;
                const int64_t q = u.q0 + wq * kQ + 16 * j + r;
                uint16_t h[8];
                __builtin_memcpy(h, __builtin_assume_aligned(turn + r * kP * 2 + (c ^ (r % kChunks)) * 16, 16), sizeof h);
                if (q < nq && p < np) {
                    const int64_t row = EPI == kBf16 && g.map ? (int64_t)g.map[g.first + q] : q;
                    uint16_t *d = out + row * ld + p;
                    if (EPI == kLogits || (aligned && p + 8 <= np)) {
                        typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
                        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, h), reinterpret_cast<u32x4 *>(d));
                    } else if (p + 8 <= np) {
                        __builtin_memcpy(d, h, sizeof h);
                    } else {
                        for (int k = 0; k < 7; ++k)
                            if (p + k < np) d[k] = h[k];
                    }
                }
            }
            asm volatile("" ::: "memory");
            __builtin_amdgcn_wave_barrier();
        };

        if constexpr (EPI == kLogits) {
            float tops[kJ], sums[kJ], hit[kJ];
            int yl[kJ];
            if (!whole)
#pragma unroll
                for (int j = 0; j < kJ; ++j)
#pragma unroll
                    for (int i = 0; i < kI; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (pw + 16 * i + r >= g.np) acc[i][j][r] = -INFINITY;
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                yl[j] = target[j] - (int)pw;
                if (yl[j] < 0 || yl[j] >= kP || yl[j] % 16 >= 4) yl[j] = -1;
                hit[j] = 0.0f;
                if (__ballot(yl[j] >= 0))
#pragma unroll
                    for (int i = 0; i < kI; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (yl[j] == 16 * i + r) hit[j] = acc[i][j][r] * kLog2e;
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < kI; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) top = fmaxf(top, acc[i][j][r]);
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                // The maximum is subtracted before the factor log2 e: its own e is then 1
                // exactly, which a product of it, rounded, would miss by 2^-24 of itself
                // (a certain row's loss would be 1e-5 for 0, on either side, at z = 250).
                const float from = top == -INFINITY ? 0.0f : top;
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < kI; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][r] - from, kLog2e, BF16 ? kScaleLog2 : 0.0f));
                        acc[i][j][r] = e;
                        sum += e;
                    }
                sum += __shfl_xor(sum, 16);
                sum += __shfl_xor(sum, 32);
                tops[j] = top * kLog2e;
                sums[j] = BF16 ? sum * 0x1p-15f : sum;
            }
            targets(unit + (int)gridDim.x);
            arrived();
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const int64_t q = qw + 16 * j;
                if (yl[j] >= 0) g.row[q].target = hit[j];
                if (q < nq && lane < 16) g.stat[q * g.subtiles + (u.p0 / kP + wp)] = f32x2{tops[j], sums[j]};
                if (!g.e) continue;
                if constexpr (BF16) {
#pragma unroll
                    for (int i = 0; i < kI; ++i) {
                        const _Float16 h[4] = {(_Float16)acc[i][j][0], (_Float16)acc[i][j][1], (_Float16)acc[i][j][2], (_Float16)acc[i][j][3]};
                        put(i, reinterpret_cast<const uint16_t *>(h));
                    }
                    send(j, static_cast<uint16_t *>(g.e), g.lde, g.lde);
                } else if (q < nq) {
#pragma unroll
                    for (int i = 0; i < kI; ++i)
                        if (pw + 16 * i < g.lde)
                            *reinterpret_cast<f32x4 *>(static_cast<float *>(g.e) + q * g.lde + pw + 16 * i) = acc[i][j];
                }
            }
        } else if (u.slot >= 0) {
            arrived();
            float *d = g.parts + (int64_t)u.slot * (BP * BQ) + (wq * kQ + lane % 16) * BP + wp * kP + lane / 16 * 4;
#pragma unroll
            for (int j = 0; j < kJ; ++j)
#pragma unroll
                for (int i = 0; i < kI; ++i) *reinterpret_cast<f32x4 *>(d + 16 * j * BP + 16 * i) = acc[i][j];
        } else {
            arrived();
            const float scale = g.sums->scale;
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const int64_t q = qw + 16 * j;
                const int64_t row = q < nq ? (g.map ? (int64_t)g.map[g.first + q] : q) : -1, at = row * g.ldo + pw;
                float *f = g.f32 + at;
                const float *fi = g.f32_in + at;
                const uint16_t *old = static_cast<const uint16_t *>(g.out) + at;
#pragma unroll
                for (int i = 0; i < kI; ++i) {
                    const int64_t here = row < 0 ? 0 : whole ? 4 : g.np - pw - 16 * i;
                    float v[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] = acc[i][j][r] * scale;
                    if (g.f32_in) {
                        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        if (here >= 4) __builtin_memcpy(x, fi + 16 * i, sizeof x);
                        else
                            for (int r = 0; r < 3; ++r)
                                if (r < here) x[r] = fi[16 * i + r];
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] += x[r];
                    }
                    if constexpr (EPI == kF32) {
                        if (here >= 4) __builtin_memcpy(f + 16 * i, v, sizeof v);
                        else
                            for (int r = 0; r < 3; ++r)
                                if (r < here) f[16 * i + r] = v[r];
                    } else {
                        uint16_t h[4] = {0, 0, 0, 0};
                        if (g.add_out) {
                            if (here >= 4) __builtin_memcpy(h, old + 16 * i, sizeof h);
                            else
                                for (int r = 0; r < 3; ++r)
                                    if (r < here) h[r] = old[16 * i + r];
#pragma unroll
                            for (int r = 0; r < 4; ++r) v[r] += widen(h[r]);
                        }
                        const uint32_t w[2] = {narrow2(v[0], v[1]), narrow2(v[2], v[3])};
                        __builtin_memcpy(h, w, sizeof h);
                        put(i, h);
                    }
                }
                if constexpr (EPI == kBf16) send(j, static_cast<uint16_t *>(g.out), g.ldo, g.np);
            }
        }
    }
}

template <bool BF16, int EPI, bool TP, bool TQ, int BP, int BQ, int WP, int WQ, int AT_ONCE, int JOIN, int DEPTH = 2>
__global__ void __launch_bounds__(64 * WP * WQ, WP * WQ == 4 && DEPTH > 2 ? 1 : 2) product_kernel(Product g) {
    product<BF16, EPI, TP, TQ, BP, BQ, WP, WQ, AT_ONCE, JOIN, DEPTH>(g);
}

// The parts of cut tiles, in order, and what a whole tile's epilogue does. Four
// rows of a tile to a workgroup.
template <int EPI>
__global__ void __launch_bounds__(256) join_kernel(Product g, int bp, int bq, int es, int at_once, int join, int part_cost) {
    const Schedule s = schedule(g, bp, bq, es, at_once, join, part_cost);
    const int per = bq / 4, tile = blockIdx.x / per;
    if (s.parts == 1 || tile >= s.cut) return;
    const int64_t nq = g.piece_is_q ? piece_rows(g.sums, g.first, g.piece) : g.nq;
    int tp, tq;
    place(s, tile, s.cut, s.whole, &tp, &tq);
    const int ql = (int)(blockIdx.x % per) * 4 + threadIdx.x / 64;
    const int64_t q = (int64_t)tq * bq + ql;
    if (q >= nq) return;
    const float scale = g.sums->scale;
    const int64_t row = g.map ? (int64_t)g.map[g.first + q] : q;
    for (int pl = threadIdx.x % 64 * 4; pl < bp; pl += 256) {
        const int64_t p = (int64_t)tp * bp + pl, left = g.np - p, at = row * g.ldo + p;
        if (left <= 0) return;
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
        for (int k = 0; k < s.parts; ++k)
            v += *reinterpret_cast<const f32x4 *>(g.parts + ((int64_t)(tile * s.parts + k) * bq + ql) * bp + pl);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (r >= left) break;
            float x = v[r] * scale;
            if (g.f32_in) x += g.f32_in[at + r];
            if (EPI == kF32) {
                g.f32[at + r] = x;
            } else {
                uint16_t *d = static_cast<uint16_t *>(g.out) + at + r;
                if (g.add_out) x += widen(*d);
                *d = (uint16_t)narrow2(x, 0.0f);
            }
        }
    }
}

// ------------------------------------------------------- e to G
// In place, [rows][vocab_p]; zeros behind the last row up to a whole stage of the
// product across the rows, and behind the vocabulary. G is rounded to the operands'
// type, as the matrix cores take it: with bf16 by up to 2^-8 of itself, which the
// products' sums average. At the target of a certain row that is -1, exact, times the
// row's weight over the largest, which is not: with weights both gradients are off by
// 2.2e-3 of their norm, without by 1.75e-3, of which 1.66e-3 is their own rounding to
// bf16. Bound by memory: 8192 rows of 50304 bf16 take 270 us (1.65 GB, 6.1 TB/s).
struct Gradient {
    const int32_t *target;        // of the piece's rows
    const f32x2 *stat;
    const HeadRow *rows;
    void *e;
    int64_t subtiles, vocab_p;
    int sub;
};

// 16 bytes of row q, from entry v on, of a piece with n rows.
template <bool BF16>
__device__ __forceinline__ void gradient_chunk(const Gradient &g, int64_t vocab, int n, int64_t q, int64_t v) {
    using T = typename Elem<BF16>::type;
    constexpr int V = 16 / sizeof(T);
    T *at = static_cast<T *>(g.e) + q * g.vocab_p + v, out[V];
    typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
    if (q < n) {
        const HeadRow s = g.rows[q];
        const int64_t y = g.target[q];
        const float share = __builtin_amdgcn_exp2f(g.stat[q * g.subtiles + v / g.sub].x - s.top) * s.inv
                            * (BF16 ? 0x1p-15f : 1.0f);
        float x[V];
        if (BF16) {
            _Float16 h[V];
            const u32x4 raw = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(at));
            __builtin_memcpy(h, &raw, sizeof h);
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = (float)h[j];
        } else {
            const u32x4 raw = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(at));
            __builtin_memcpy(x, &raw, sizeof x);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] *= share;
        if (y >= v && y < v + V)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (v + j == y) x[j] -= s.share;
        if (v + V > vocab)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (v + j >= vocab) x[j] = 0.0f;
        if constexpr (BF16) {
            uint32_t w[V / 2];
#pragma unroll
            for (int j = 0; j < V / 2; ++j) w[j] = narrow2(x[2 * j], x[2 * j + 1]);
            __builtin_memcpy(out, w, sizeof out);
        } else {
            __builtin_memcpy(out, x, sizeof out);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] = 0;
    }
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, out), reinterpret_cast<u32x4 *>(at));
}

template <bool BF16>
__global__ void __launch_bounds__(256)
gradient_kernel(Gradient g, int64_t vocab, const HeadSums *sums, int64_t first, int64_t piece, uint32_t per_row) {
    constexpr int V = BF16 ? 8 : 4;
    const int n = piece_rows(sums, first, piece);
    const int64_t q = blockIdx.x / per_row, v = ((int64_t)(blockIdx.x % per_row) * 256 + threadIdx.x) * V;
    if (q < round_up(n, 64) && v < g.vocab_p) gradient_chunk<BF16>(g, vocab, n, q, v);
}

// ------------------------------------------------------- the softmax
// LANES of a wave: the maximum and sum of row q of the piece from its tiles', and
// its loss.
template <int LANES>
__device__ __forceinline__ void softmax_row(const HeadArgs &a, const HeadSums *sums, const int32_t *map, int64_t first,
                                            const f32x2 *stat, int64_t subtiles, HeadRow *rows, float *losses, int64_t q, int lane) {
    const f32x2 *s = stat + q * subtiles;
    float top = -INFINITY;
    for (int64_t k = lane; k < subtiles; k += LANES) top = fmaxf(top, s[k].x);
    for (int d = LANES / 2; d; d /= 2) top = fmaxf(top, __shfl_xor(top, d));
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    for (int64_t k = lane; k < subtiles; k += LANES) sum += s[k].y * __builtin_amdgcn_exp2f(s[k].x - base);
    for (int d = LANES / 2; d; d /= 2) sum += __shfl_xor(sum, d);
    if (lane) return;
    const int64_t i = map[first + q];
    const float w = a.weights ? a.weights[i] : 1.0f;
    const float share = w / sums->most;
    // Not negative: top >= target, since both are rounded the same way (0 where the
    // target is the largest), and sum >= 1, since the largest entry's e is 1.
    losses[i] = (float)(((double)(base - rows[q].target) + (double)__builtin_amdgcn_logf(sum)) * kLn2);
    rows[q].top = base;
    rows[q].inv = share / sum;
    rows[q].share = share;
}

__global__ void __launch_bounds__(256)
softmax_kernel(HeadArgs a, const HeadSums *sums, const int32_t *map, int64_t first, int64_t piece,
               const f32x2 *stat, int64_t subtiles, HeadRow *rows, float *losses) {
    const int64_t q = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
    if (q < piece_rows(sums, first, piece))
        softmax_row<64>(a, sums, map, first, stat, subtiles, rows, losses, q, threadIdx.x % 64);
}

// One workgroup: the weighted sum of the losses, in binary64; in small calls of the
// rows' softmax first, and of e's turning into G (g.e, if there).
template <bool BF16>
__global__ void __launch_bounds__(1024)
loss_kernel(HeadArgs a, const HeadSums *sums, const int32_t *map, Gradient g, HeadRow *rows, float *losses) {
    __shared__ double parts[16];
    if (g.stat) {
        const int n = (int)sums->rows;
        if (g.subtiles <= kFewStats)
            for (int64_t q = threadIdx.x / 16; q < n; q += 64)
                softmax_row<16>(a, sums, map, 0, g.stat, g.subtiles, rows, losses, q, threadIdx.x % 16);
        else
            for (int64_t q = threadIdx.x / 64; q < n; q += 16)
                softmax_row<64>(a, sums, map, 0, g.stat, g.subtiles, rows, losses, q, threadIdx.x % 64);
        __syncthreads();                          // a workgroup sees its own stores
        constexpr int V = BF16 ? 8 : 4;
        const uint32_t per_row = (uint32_t)(g.vocab_p / V);
        if (g.e)
            for (uint32_t k = threadIdx.x; k < (uint32_t)round_up(n, 64) * per_row; k += 1024)
                gradient_chunk<BF16>(g, a.vocab, n, k / per_row, (int64_t)(k % per_row) * V);
    }
    double sum = 0.0;
    const int64_t rows_in = sums->rows;
#pragma unroll 8
    for (int64_t k = threadIdx.x; k < rows_in; k += 1024) {
        const int64_t i = map[k];
        sum += (a.weights ? (double)a.weights[i] : 1.0) * (double)losses[i];
    }
    for (int s = 32; s; s /= 2) sum += __shfl_xor(sum, s);
    if (threadIdx.x % 64 == 0) parts[threadIdx.x / 64] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.0;
        for (int w = 0; w < 16; ++w) sum += parts[w];
        *a.loss = (float)(a.mean && sums->weight != 0.0 ? sum / sums->weight : sum);
    }
}

// Rows of grad_hidden that take no part: zero.
__global__ void __launch_bounds__(256) idle_rows_kernel(HeadArgs a) {
    for (int64_t i = (int64_t)blockIdx.x * 4 + threadIdx.x / 64; i < a.count; i += (int64_t)gridDim.x * 4)
        if (!takes_part(a, i)) idle_row(a, i, threadIdx.x % 64);
}

// ------------------------------------------------------- launches
template <bool BF16, int EPI, bool TP, bool TQ>
void start_product(const Product &g, int shape, hipStream_t stream) {
    const TileShape t = kTiles[shape];
    const int64_t tiles = ceil_div(g.np, t.p) * ceil_div(g.nq, t.q);
    const unsigned grid = (unsigned)(g.slots > 0 || tiles > t.at_once ? t.at_once : tiles);
    if constexpr (EPI == kLogits) {
        if constexpr (BF16) {
            if (shape == 3) product_kernel<BF16, EPI, TP, TQ, 128, 32, 4, 1, 256, 1, 4><<<grid, 256, 0, stream>>>(g);
            if (shape == 4) product_kernel<BF16, EPI, TP, TQ, 128, 64, 4, 2, 256, 1, 4><<<grid, 512, 0, stream>>>(g);
            if (shape == 5) product_kernel<BF16, EPI, TP, TQ, 128, 128, 2, 4, 256, 1, 4><<<grid, 512, 0, stream>>>(g);
            if (shape == 6) product_kernel<BF16, EPI, TP, TQ, 128, 192, 2, 4, 256, 1, 3><<<grid, 512, 0, stream>>>(g);
            if (shape == 7) product_kernel<BF16, EPI, TP, TQ, 128, 256, 2, 4, 256, 1, 3><<<grid, 512, 0, stream>>>(g);
        }
    }
    if constexpr (BF16)
        if (shape == 0) product_kernel<BF16, EPI, TP, TQ, 256, 256, 2, 4, kTiles[0].at_once, BF16 ? kTiles[0].join : 4 * kTiles[0].join><<<grid, 512, 0, stream>>>(g);
    if (shape == 1) product_kernel<BF16, EPI, TP, TQ, 128, 128, 2, 2, kTiles[1].at_once, BF16 ? kTiles[1].join : 4 * kTiles[1].join><<<grid, 256, 0, stream>>>(g);
    if (shape == 2) product_kernel<BF16, EPI, TP, TQ, 128, 32, 4, 1, kTiles[2].at_once, BF16 ? kTiles[2].join : 4 * kTiles[2].join><<<grid, 256, 0, stream>>>(g);
    if constexpr (EPI != kLogits)
        if (g.slots > 0) {
            const int64_t cut = tiles < t.at_once ? tiles : t.at_once - 1;
            join_kernel<EPI><<<(unsigned)(cut * (t.q / 4)), 256, 0, stream>>>(g, t.p, t.q, BF16 ? 2 : 4, t.at_once, BF16 ? t.join : 4 * t.join, BF16 ? kPartCost16 : kPartCost32);
        }
}

template <bool BF16>
hipError_t head(const HeadArgs &a, const HeadPlan &p, hipStream_t stream) {
    char *w = a.workspace;
    const int es = BF16 ? 2 : 4;
    auto *sums = reinterpret_cast<HeadSums *>(w + p.sum_off);
    auto *map = reinterpret_cast<int32_t *>(w + p.map_off), *target = map + a.count;
    auto *losses = a.losses ? a.losses : reinterpret_cast<float *>(w + p.loss_off);
    auto *rows = reinterpret_cast<HeadRow *>(w + p.row_off);
    auto *stat = reinterpret_cast<f32x2 *>(w + p.stat_off);
    const bool grads = a.grad_hidden || a.grad_table;
    void *packed = p.pack_with_rows ? w + p.hidden_off : nullptr;
    if (a.count <= 2048) rows_kernel<BF16, 1><<<1, 1024, 0, stream>>>(a, sums, map, target, losses, p.idle_with_rows, packed, p.width_p);
    else rows_kernel<BF16, 8><<<1, 1024, 0, stream>>>(a, sums, map, target, losses, p.idle_with_rows, packed, p.width_p);
    if (a.grad_hidden && !p.idle_with_rows) idle_rows_kernel<<<(unsigned)(a.count < 65536 ? ceil_div(a.count, 4) : 16384), 256, 0, stream>>>(a);
    const void *table = a.table;
    if (p.pack_table) {
        pack_table_kernel<BF16><<<(unsigned)a.vocab, 256, 0, stream>>>(a, w + p.table_off, p.width_p);
        table = w + p.table_off;
    }
    for (int64_t k = 0; k < p.pieces; ++k) {
        const int64_t first = k * p.piece;
        if (!p.pack_with_rows)
            pack_hidden_kernel<BF16><<<(unsigned)p.piece_p, 256, 0, stream>>>(a, map, sums, first, p.piece, w + p.hidden_off, p.width_p);
        Product g = {};
        g.sums = sums;
        g.first = first;
        g.piece = p.piece;
        g.p = table;
        g.ldp = p.width_p * es;
        g.np = a.vocab;
        g.q = w + p.hidden_off;
        g.ldq = p.width_p * es;
        g.nq = p.piece;
        g.piece_is_q = true;
        g.steps = p.width_p * es / 128;
        g.target = target;
        g.stat = stat;
        g.row = rows;
        g.subtiles = p.subtiles;
        g.e = grads ? w + p.e_off : nullptr;
        g.lde = p.vocab_p;
        start_product<BF16, kLogits, false, false>(g, p.tile_logits, stream);
        Gradient turned = {target + first, stat, rows, w + p.e_off, p.subtiles, p.vocab_p, p.sub};
        if (p.softmax_with_loss) {
            if (!p.turn_with_loss) turned.e = nullptr;
            loss_kernel<BF16><<<1, 1024, 0, stream>>>(a, sums, map, turned, rows, losses);
            turned.e = w + p.e_off;
        } else {
            softmax_kernel<<<(unsigned)ceil_div(p.piece, 4), 256, 0, stream>>>(a, sums, map, first, p.piece, stat, p.subtiles,
                                                                               rows, losses);
        }
        if (!grads) continue;
        if (!p.turn_with_loss) {
            const int64_t per_row = ceil_div(p.vocab_p * es, 256 * 16);
            gradient_kernel<BF16><<<(unsigned)(p.piece_p * per_row), 256, 0, stream>>>(turned, a.vocab, sums, first, p.piece, (uint32_t)per_row);
        }
        if (a.grad_hidden) {
            Product h = {};
            h.sums = sums;
            h.first = first;
            h.piece = p.piece;
            h.p = table;
            h.ldp = p.width_p * es;
            h.kp = a.vocab;
            h.np = a.width;
            h.q = w + p.e_off;
            h.ldq = p.vocab_p * es;
            h.nq = p.piece;
            h.piece_is_q = true;
            h.steps = ceil_div(a.vocab * es, 128);    // every stage has a row of the table
            h.ldo = a.width;
            h.slots = p.slots_hidden;
            h.parts = reinterpret_cast<float *>(w + p.parts_off);
            h.map = map;
            h.out = a.grad_hidden;
            h.f32 = static_cast<float *>(a.grad_hidden);
            start_product<BF16, BF16 ? kBf16 : kF32, true, false>(h, p.tile_hidden, stream);
        }
        if (a.grad_table) {
            Product t = {};
            t.sums = sums;
            t.first = first;
            t.piece = p.piece;
            t.p = w + p.hidden_off;
            t.ldp = p.width_p * es;
            t.kp = t.kq = p.piece_p;
            t.np = a.width;
            t.q = w + p.e_off;
            t.ldq = p.vocab_p * es;
            t.nq = a.vocab;
            t.piece_is_k = true;
            t.ldo = a.width;
            const bool last = k + 1 == p.pieces;
            float *gw = a.table_grad_bf16 ? reinterpret_cast<float *>(w + p.gw_off) : static_cast<float *>(a.grad_table);
            t.slots = p.slots_table;
            t.parts = reinterpret_cast<float *>(w + p.parts_off);
            t.f32_in = k > 0 || (!a.table_grad_bf16 && a.accumulate) ? gw : nullptr;
            if (a.table_grad_bf16 && last) {
                t.out = a.grad_table;
                t.add_out = a.accumulate;
                start_product<BF16, kBf16, true, true>(t, p.tile_table, stream);
            } else {
                t.f32 = gw;
                start_product<BF16, kF32, true, true>(t, p.tile_table, stream);
            }
        }
    }
    if (!p.softmax_with_loss) loss_kernel<BF16><<<1, 1024, 0, stream>>>(a, sums, map, Gradient{}, rows, losses);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_head(const HeadArgs &a, const HeadPlan &p, hipStream_t stream) {
    return a.bf16 ? head<true>(a, p, stream) : head<false>(a, p, stream);
}

}  // namespace zk
