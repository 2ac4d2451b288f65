// Softmax cross entropy of hidden states against a vocabulary table, with the
// gradients of both, for gfx950.
//
//   z_iv = h_i . W_v,  l_i = log sum_v exp(z_iv) - z_iy
//   G_iv = w_i (exp(z_iv) / sum_u exp(z_iu) - [v = y]),  dh_i = s sum_v G_iv W_v,
//   dW_v = s sum_i G_iv h_i
//
// Three products of rows with rows (both operands' long axis contiguous) on the
// matrix cores, tile by tile through LDS. The first one's epilogue takes each
// tile's maximum and sum of exponentials per row, in binary32 from the
// accumulators, and leaves e = exp(z - its tile's maximum) instead of z: e needs
// 2 bytes where z would need 4 for the same p, for e's relative error is p's.
// With the row's maximum and sum known, one pass turns e into G, the operand of
// the other two products. w are the weights over the largest, and s the rest of
// the gradient's scale, which multiplies the products' binary32 sums: rounded to
// bf16 with s inside, the -s of the many entries with p = 0 would all be off by
// the same; so they are -1 and exact. Rows that take
// no part (target outside the table, weight 0) are left out of all products.
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

__device__ __forceinline__ uint16_t narrow(float f) {
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);
    return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
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
    return (int)(n < 0 ? 0 : n < piece ? n : piece);
}

// ------------------------------------------------------- which rows
// One workgroup: the rows that take part, in order, with their targets, and
// their weights' sum.
__global__ void __launch_bounds__(1024) rows_kernel(HeadArgs a, HeadSums *sums, int32_t *map, int32_t *target) {
    __shared__ int32_t found[16];
    __shared__ double parts[16];
    __shared__ float tops[16];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    int64_t base = 0;
    double weight = 0.0;
    float most = 0.0f;
    for (int64_t i0 = 0; i0 < a.count; i0 += 1024) {
        const int64_t i = i0 + threadIdx.x;
        bool on = false;
        if (i < a.count) {
            on = takes_part(a, i);
            if (on) {
                const float w = a.weights ? a.weights[i] : 1.0f;
                weight += (double)w;
                most = fmaxf(most, fabsf(w));
            }
        }
        const uint64_t mask = __ballot(on);
        if (lane == 0) found[wave] = __popcll(mask);
        __syncthreads();
        int64_t at = base;
        for (int w = 0; w < 16; ++w) {
            if (w < wave) at += found[w];
            base += found[w];
        }
        if (on) {
            at += __popcll(mask & ((1ull << lane) - 1));
            map[at] = (int32_t)i;
            target[at] = (int32_t)load_id(a.targets, a.wide_ids, i);
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
}

// ------------------------------------------------------- copies
// dst [rows_p][cols_p] = the mapped rows of src [.][cols], zeros behind them.
// A row of threads to a destination row.
template <bool BF16>
__global__ void __launch_bounds__(256)
pack_kernel(const void *src, int64_t rows, int64_t cols, const int32_t *map, const HeadSums *sums,
            int64_t first, void *dst, int64_t rows_p, int64_t cols_p) {
    using T = typename Elem<BF16>::type;
    const int64_t r = blockIdx.x;
    const int64_t n = map ? piece_rows(sums, first, rows) : rows;
    if (r >= n && r >= round_up(n, 64)) return;
    const int64_t from = r < n ? (map ? map[first + r] : r) : -1;
    const T *s = static_cast<const T *>(src) + from * cols;
    T *d = static_cast<T *>(dst) + r * cols_p;
    constexpr int V = 16 / sizeof(T);
    for (int64_t c = (int64_t)threadIdx.x * V; c < cols_p; c += 256 * V) {
        T x[V];
        if (from >= 0 && c + V <= cols) {
            __builtin_memcpy(x, s + c, sizeof x);
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) x[k] = from >= 0 && c + k < cols ? s[c + k] : (T)0;
        }
        __builtin_memcpy(__builtin_assume_aligned(d + c, 16), x, sizeof x);
    }
}

// ------------------------------------------------------- the product
// out[q][p] = sum_k P[p][k] Q[q][k]; rows of P and Q are 16-byte aligned and
// their long axis is a whole number of 128-byte steps. A workgroup makes BP x BQ
// outputs with WP x WQ waves; a step of both operands' rows, 128 bytes each, goes
// straight from memory to LDS while the step before it is multiplied.
//
// LDS holds a row's 128 bytes as eight 16-byte chunks, chunk c at place
// c ^ (row % 8): then the 16 rows that a fragment reads at one chunk lie on
// different banks. A load to LDS writes lane after lane, so the exchange is made
// in the addresses it reads from.

enum Epilogue { kLogits, kBf16, kF32 };

struct Product {
    const void *p, *q;
    int64_t ldp, ldq;             // bytes
    int64_t np, nq;               // rows
    int64_t steps;                // of 128 bytes on the long axis
    int tiles_p, tiles_q, splits;
    // with sums: rows of the piece, which bound nq or the long axis
    const HeadSums *sums;
    int64_t first, piece;
    bool piece_is_q, piece_is_k;
    int64_t kp;                   // lines of a P across the long axis
    // kLogits
    const int32_t *target;        // of the rows of Q
    f32x2 *stat;
    HeadRow *row;
    int64_t subtiles;
    void *e;                      // null: not wanted
    int64_t lde;                  // elements
    const int32_t *map;           // rows of the output, if they are others
    // kBf16: out = scaled product + f32_in + old out; kF32: f32 = scaled product + f32_in
    float *f32;
    int64_t f32_split;            // elements between splits
    const float *f32_in;          // or null
    void *out;
    bool add_out;
    int64_t ldo;                  // elements, of f32, f32_in and out
};

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

// 16 bytes a lane, from base + from, to LDS at `lds` + 16 * lane. In assembly,
// since the compiler would otherwise wait for all such loads before it reads LDS
// across lanes (ds_read_b64_tr_b16); the waits are the loop's own. No register is
// written.
__device__ __forceinline__ void load_to_lds(const char *base, int from, uint32_t lds) {
    typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
    const u32x4 r = {(uint32_t)(uintptr_t)base, (uint32_t)((uintptr_t)base >> 32) & 0xFFFFu, 0xFFFFFFFFu, 0x00027000u};
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(from), "s"(r)
                 : "memory");
}

// One operand's tile of a stage: B rows and 128 bytes of the long axis, from
// rows along it ([row][k], T false) or across it ([k][row], T true).
template <bool BF16, bool T, int B, int LOADS>
struct Operand {
    static constexpr int kEs = BF16 ? 2 : 4, kSteps = 128 / kEs;
    static constexpr int kLine = T ? B * kEs : 128;           // bytes of a line in LDS
    int at[LOADS];                                            // what each load's lane reads
    int64_t step;                                             // bytes from stage to stage

    // Where the 16-byte chunk at place c of line k comes from.
    static __device__ __forceinline__ int source(int k, int c) {
        if (!T) return c ^ (k % 8);
        if (BF16) return c ^ ((((k & 3) | ((k >> 1) & 4)) << 1) & (kLine / 16 - 1));
        return c ^ (((k >> 2) & 3) << 2 & (kLine / 16 - 1));
    }
    // Rows (T: 16-byte columns) behind the operand's last are read as the last:
    // always memory of the operand.
    __device__ __forceinline__ void init(int wave, int lane, int64_t first, int64_t n, int64_t ld) {
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            const int byte = (wave * LOADS + j) * 1024 + lane * 16;
            const int line = byte / kLine, chunk = source(line, byte % kLine / 16);
            if (T) {
                int64_t col = first * kEs + chunk * 16;
                if (col > ld - 16) col = ld - 16;
                at[j] = (int)(line * ld + (col - first * kEs));
            } else {
                int64_t r = line;
                if (first + r >= n) r = n - 1 - first;
                at[j] = (int)(r * ld) + chunk * 16;
            }
        }
        step = T ? kSteps * ld : 128;
    }
    // lds: the operand's place in the stage. T: of a stage with fewer than
    // kSteps lines (`left` >= 1) those behind are read as the last.
    template <bool LAST>
    __device__ __forceinline__ void load(const char *base, uint32_t lds, int wave, int lane, int left, int ld) const {
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            int from = at[j];
            if (LAST) {
                const int line = ((wave * LOADS + j) * 1024 + lane * 16) / kLine;
                if (line >= left) from -= (line - (left - 1)) * ld;
            }
            load_to_lds(base, from, lds + (wave * LOADS + j) * 1024);
        }
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

template <bool BF16, int EPI, bool TP, bool TQ, int BP, int BQ, int WP, int WQ>
__device__ __forceinline__ void product(const Product &g) {
    constexpr int kWaves = WP * WQ;
    constexpr int kI = BP / WP / 16, kJ = BQ / WQ / 16;       // fragments of a wave
    constexpr int kLoadsP = BP / 8 / kWaves, kLoadsQ = BQ / 8 / kWaves;
    static_assert(kLoadsP * 8 * kWaves == BP && kLoadsQ * 8 * kWaves == BQ, "whole loads");
    constexpr int kStage = (BP + BQ) * 128;
    using F = typename Frag<BF16>::type;
    using OpP = Operand<BF16, TP, BP, kLoadsP>;
    using OpQ = Operand<BF16, TQ, BQ, kLoadsQ>;
    constexpr int kOut = EPI != kF32 ? BQ * (2 * BP + 16) : 0;
    __shared__ __align__(1024) char lds[2 * kStage > kOut ? 2 * kStage : kOut];

    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    int64_t nq = g.nq, steps = g.steps;
    if (g.sums) {
        const int n = piece_rows(g.sums, g.first, g.piece);
        if (g.piece_is_q) nq = n;
        if (g.piece_is_k) steps = ceil_div((int64_t)n * OpP::kEs, 128);
    }

    // Workgroups go round robin over the 8 XCDs: give each XCD a run of
    // neighbouring tiles, in groups of 8 along p, so that its L2 is shared.
    const int tiles = g.tiles_p * g.tiles_q;
    const int split = blockIdx.x / tiles;
    int t = blockIdx.x % tiles;
    {
        const int per = tiles / 8, rest = tiles % 8, x = t % 8;
        t = x * per + (x < rest ? x : rest) + t / 8;
    }
    const int group = t / (8 * g.tiles_q), in = t % (8 * g.tiles_q);
    const int gp = g.tiles_p - 8 * group < 8 ? g.tiles_p - 8 * group : 8;
    const int64_t p0 = (int64_t)(8 * group + in % gp) * BP, q0 = (int64_t)(in / gp) * BQ;
    if (q0 >= nq) return;
    const int64_t per_split = ceil_div(steps, g.splits);
    const int64_t k0 = per_split * split;
    const int ksteps = (int)(k0 >= steps ? 0 : steps - k0 < per_split ? steps - k0 : per_split);

    OpP op;
    OpQ oq;
    op.init(wave, lane, p0, g.np, g.ldp);
    oq.init(wave, lane, q0, nq, g.ldq);
    const char *bp = static_cast<const char *>(g.p) + (TP ? p0 * OpP::kEs : p0 * g.ldp) + k0 * op.step;
    const char *bq = static_cast<const char *>(g.q) + (TQ ? q0 * OpQ::kEs : q0 * g.ldq) + k0 * oq.step;
    // lines of P that are left (TP: the table's rows are not padded)
    int64_t lines = TP ? g.kp - k0 * OpP::kSteps : 0;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void *)lds);

    auto load = [&](int buf) {
        const uint32_t s = lds0 + buf * kStage;
        if (TP && lines < OpP::kSteps) op.template load<true>(bp, s, wave, lane, (int)lines, (int)g.ldp);
        else op.template load<false>(bp, s, wave, lane, 0, 0);
        oq.template load<false>(bq, s + BP * 128, wave, lane, 0, 0);
        bp += op.step;
        bq += oq.step;
        lines -= OpP::kSteps;
    };

    int target[kJ];
    if constexpr (EPI == kLogits)
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const int64_t q = q0 + wave % WQ * (BQ / WQ) + lane % 16 + 16 * j;
            target[j] = q < nq ? g.target[g.first + q] : -1;
        }

    f32x4 acc[kI][kJ];
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int j = 0; j < kJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // A stage is multiplied in four parts: part c takes half c / 2 of the long axis
    // and half c % 2 of the wave's rows of P.
    const int wp = wave / WQ, wq = wave % WQ;
    F fp[2][kI / 2], fq[2][kJ];
    auto read = [&](int buf, int c) {
        const char *s = lds + buf * kStage;
        if (c % 2 == 0)
#pragma unroll
            for (int j = 0; j < kJ; ++j) fq[c / 2][j] = OpQ::read(s + BP * 128, wq * (BQ / WQ) + 16 * j, c / 2, lane);
#pragma unroll
        for (int i = 0; i < kI / 2; ++i)
            fp[c % 2][i] = OpP::read(s, wp * (BP / WP) + 16 * (c % 2 * (kI / 2) + i), c / 2, lane);
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

    // Each part is read while the one before is multiplied. When the last part of a
    // stage has been read by all, the loads of the stage after the next go to its
    // place, so a load has nearly a stage's time to arrive and a wave meets one
    // barrier a stage, with products still to do.
    if (ksteps > 0) load(0);
    if (ksteps > 1) load(1);
    if (ksteps > 1) asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" : : "n"(kLoadsP + kLoadsQ) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    if (ksteps > 0) read(0, 0);
    for (int k = 0; k < ksteps; ++k) {
        const int buf = k & 1;
        read(buf, 1);
        __builtin_amdgcn_sched_barrier(0);        // the reads go first, whatever the scheduler thinks
        multiply(0);
        __builtin_amdgcn_sched_barrier(0);
        read(buf, 2);
        __builtin_amdgcn_sched_barrier(0);
        multiply(1);
        __builtin_amdgcn_sched_barrier(0);
        read(buf, 3);
        __builtin_amdgcn_sched_barrier(0);
        multiply(2);
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (k + 2 < ksteps) load(buf);
        if (k + 1 < ksteps) read(buf ^ 1, 0);
        __builtin_amdgcn_sched_barrier(0);
        multiply(3);
    }

    // A lane holds outputs p = pw + 16 i + r, r < 4, of q = qw + 16 j.
    const int pl = wp * (BP / WP) + lane / 16 * 4, ql = wq * (BQ / WQ) + lane % 16;
    const int64_t pw = p0 + pl, qw = q0 + ql;
    const bool whole = p0 + BP <= g.np;
    // Numbers of two bytes go out through LDS, [q][p], for whole lines: a lane's
    // four are 8 bytes of a line, 16 lines to an instruction. 16 bytes between
    // rows keep the 16 on different banks.
    constexpr int kPitch = 2 * BP + 16;
    auto put = [&](int i, int j, const uint16_t *h) {
        __builtin_memcpy(__builtin_assume_aligned(lds + (ql + 16 * j) * kPitch + (pl + 16 * i) * 2, 8), h, 8);
    };
    if constexpr (EPI == kLogits) {
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const int64_t q = qw + 16 * j;
            const bool on = q < nq;
            if (!whole)
#pragma unroll
                for (int i = 0; i < kI; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (pw + 16 * i + r >= g.np) acc[i][j][r] = -INFINITY;
            const int yl = target[j] - (int)pw;
            if (__ballot(yl >= 0 && yl < BP / WP && yl % 16 < 4))
#pragma unroll
                for (int i = 0; i < kI; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (yl == 16 * i + r) g.row[q].target = acc[i][j][r] * kLog2e;
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < kI; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) top = fmaxf(top, acc[i][j][r]);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32)) * kLog2e;
            const float base = (BF16 ? kScaleLog2 : 0.0f) - (top == -INFINITY ? 0.0f : top);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kI; ++i) {
                float e[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    e[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][r], kLog2e, base));
                    sum += e[r];
                }
                if (!g.e) continue;
                if constexpr (BF16) {
                    const _Float16 h[4] = {(_Float16)e[0], (_Float16)e[1], (_Float16)e[2], (_Float16)e[3]};
                    put(i, j, reinterpret_cast<const uint16_t *>(h));
                } else if (on && pw + 16 * i < g.lde) {
                    *reinterpret_cast<f32x4 *>(static_cast<float *>(g.e) + q * g.lde + pw + 16 * i) = f32x4{e[0], e[1], e[2], e[3]};
                }
            }
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (on && lane < 16)
                g.stat[q * g.subtiles + (p0 / (BP / WP) + wp)] = f32x2{top, BF16 ? sum * 0x1p-15f : sum};
        }
    } else {
        const float scale = g.sums->scale;
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const int64_t q = qw + 16 * j;
            if (EPI == kF32 && q >= nq) continue;
            const int64_t row = q < nq ? (g.map ? (int64_t)g.map[g.first + q] : q) : -1, at = row * g.ldo + pw;
            float *f = g.f32 + split * g.f32_split + at;
            const float *fi = g.f32_in + at;
            const uint16_t *old = static_cast<const uint16_t *>(g.out) + at;
#pragma unroll
            for (int i = 0; i < kI; ++i) {
                const int64_t left = row < 0 ? 0 : whole ? 4 : g.np - pw - 16 * i;
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = acc[i][j][r] * scale;
                if (g.f32_in) {
                    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    if (left >= 4) __builtin_memcpy(x, fi + 16 * i, sizeof x);
                    else
                        for (int r = 0; r < 3; ++r)
                            if (r < left) x[r] = fi[16 * i + r];
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] += x[r];
                }
                if constexpr (EPI == kF32) {
                    if (left >= 4) __builtin_memcpy(f + 16 * i, v, sizeof v);
                    else
                        for (int r = 0; r < 3; ++r)
                            if (r < left) f[16 * i + r] = v[r];
                } else {
                    uint16_t h[4] = {0, 0, 0, 0};
                    if (g.add_out) {
                        if (left >= 4) __builtin_memcpy(h, old + 16 * i, sizeof h);
                        else
                            for (int r = 0; r < 3; ++r)
                                if (r < left) h[r] = old[16 * i + r];
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] += widen(h[r]);
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) h[r] = narrow(v[r]);
                    put(i, j, h);
                }
            }
        }
    }
    if constexpr (EPI == kBf16 || (EPI == kLogits && BF16)) {
        if (EPI == kLogits && !g.e) return;
        __syncthreads();
        constexpr int kAcross = BP / 8, kDown = 64 * kWaves / kAcross;    // 16-byte chunks of a line; lines at a time
        const int64_t p = p0 + threadIdx.x % kAcross * 8;
        const int64_t np = EPI == kLogits ? g.lde : g.np, ld = EPI == kLogits ? g.lde : g.ldo;
        uint16_t *out = static_cast<uint16_t *>(EPI == kLogits ? g.e : g.out);
        if (p >= np) return;
#pragma unroll 4
        for (int r = threadIdx.x / kAcross; r < BQ; r += kDown) {
            if (q0 + r >= nq) break;
            const int64_t row = EPI == kBf16 && g.map ? (int64_t)g.map[g.first + q0 + r] : q0 + r;
            uint16_t h[8], *d = out + row * ld + p;
            __builtin_memcpy(h, __builtin_assume_aligned(lds + r * kPitch + threadIdx.x % kAcross * 16, 16), sizeof h);
            if (p + 8 <= np) __builtin_memcpy(d, h, sizeof h);
            else
                for (int k = 0; k < 7; ++k)
                    if (p + k < np) d[k] = h[k];
        }
    }
}

template <bool BF16, int EPI, bool TP, bool TQ, int BP, int BQ, int WP, int WQ>
__global__ void __launch_bounds__(64 * WP * WQ, 2) product_kernel(Product g) {
    product<BF16, EPI, TP, TQ, BP, BQ, WP, WQ>(g);
}

// ------------------------------------------------------- the softmax
// A wave to a row: its maximum and sum from its tiles', and its loss.
__global__ void __launch_bounds__(256)
softmax_kernel(HeadArgs a, const HeadSums *sums, const int32_t *map, int64_t first, int64_t piece,
               const f32x2 *stat, int64_t subtiles, HeadRow *rows, float *losses) {
    const int lane = threadIdx.x % 64;
    const int64_t q = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
    if (q >= piece_rows(sums, first, piece)) return;
    const f32x2 *s = stat + q * subtiles;
    float top = -INFINITY;
    for (int64_t k = lane; k < subtiles; k += 64) top = fmaxf(top, s[k].x);
    for (int d = 32; d; d /= 2) top = fmaxf(top, __shfl_xor(top, d));
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    for (int64_t k = lane; k < subtiles; k += 64) sum += s[k].y * __builtin_amdgcn_exp2f(s[k].x - base);
    for (int d = 32; d; d /= 2) sum += __shfl_xor(sum, d);
    if (lane) return;
    const int64_t i = map[first + q];
    const float w = a.weights ? a.weights[i] : 1.0f;
    const float share = w / sums->most;
    // top - target first: exact where the target is the largest, which is where
    // the loss is small
    losses[i] = (float)(((double)(base - rows[q].target) + (double)__builtin_amdgcn_logf(sum)) * kLn2);
    rows[q].top = base;
    rows[q].inv = share / sum;
    rows[q].share = share;
}

// One workgroup: the weighted sum of the losses, in binary64.
__global__ void __launch_bounds__(1024)
loss_kernel(HeadArgs a, const HeadSums *sums, const int32_t *map, const float *losses) {
    __shared__ double parts[16];
    double sum = 0.0;
    for (int64_t k = threadIdx.x; k < sums->rows; k += 1024) {
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

// losses and rows of grad_hidden that take no part: zero.
__global__ void __launch_bounds__(256) idle_rows_kernel(HeadArgs a, float *losses) {
    const int lane = threadIdx.x % 64;
    const int64_t i = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
    if (i >= a.count) return;
    if (takes_part(a, i)) return;
    if (lane == 0) losses[i] = 0.0f;
    if (!a.grad_hidden) return;
    for (int64_t c = lane; c < a.width; c += 64)
        if (a.bf16) static_cast<uint16_t *>(a.grad_hidden)[i * a.width + c] = 0;
        else static_cast<float *>(a.grad_hidden)[i * a.width + c] = 0.0f;
}

// ------------------------------------------------------- e to G
// In place, [rows][vocab_p]; zeros behind the last row up to a whole stage of the
// product across the rows, and behind the vocabulary. Eight (four) numbers to a
// thread, grid (columns, rows).
template <bool BF16>
__global__ void __launch_bounds__(256)
gradient_kernel(HeadArgs a, const HeadSums *sums, const int32_t *target, int64_t first, int64_t piece,
                const f32x2 *stat, int64_t subtiles, int sub, const HeadRow *rows, void *e,
                int64_t vocab_p) {
    using T = typename Elem<BF16>::type;
    constexpr int V = 16 / sizeof(T);
    const int n = piece_rows(sums, first, piece);
    const int64_t q = blockIdx.y, v = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
    if (q >= round_up(n, 64) || v >= vocab_p) return;
    T *at = static_cast<T *>(e) + q * vocab_p + v, out[V];
    if (q < n) {
        const HeadRow s = rows[q];
        const int64_t y = target[first + q];
        const float share = __builtin_amdgcn_exp2f(stat[q * subtiles + v / sub].x - s.top) * s.inv
                            * (BF16 ? 0x1p-15f : 1.0f);
        float x[V];
        if (BF16) {
            _Float16 h[V];
            __builtin_memcpy(h, __builtin_assume_aligned(at, 16), sizeof h);
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = (float)h[j];
        } else {
            __builtin_memcpy(x, __builtin_assume_aligned(at, 16), sizeof x);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float d = x[j] * share;
            if (v + j == y) d -= s.share;
            if (v + j >= a.vocab) d = 0.0f;
            if constexpr (BF16) out[j] = narrow(d);
            else out[j] = d;
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] = 0;
    }
    __builtin_memcpy(__builtin_assume_aligned(at, 16), out, sizeof out);
}

// grad_hidden from the binary32 parts of the split product.
template <bool BF16>
__global__ void __launch_bounds__(256)
join_kernel(HeadArgs a, const HeadSums *sums, const int32_t *map, int64_t first, int64_t piece,
            const float *parts, int splits, int64_t stride) {
    const int64_t q = blockIdx.x;
    if (q >= piece_rows(sums, first, piece)) return;
    const int64_t row = map[first + q];
    for (int64_t c = threadIdx.x; c < a.width; c += 256) {
        float v = 0.0f;
        for (int s = 0; s < splits; ++s) v += parts[s * stride + q * a.width + c];
        if (BF16) static_cast<uint16_t *>(a.grad_hidden)[row * a.width + c] = narrow(v);
        else static_cast<float *>(a.grad_hidden)[row * a.width + c] = v;
    }
}

// ------------------------------------------------------- launches
template <bool BF16, int EPI, bool TP, bool TQ>
void start_product(const Product &g, int shape, hipStream_t stream) {
    const dim3 grid((unsigned)(g.tiles_p * g.tiles_q * g.splits));
    if (shape == 0) product_kernel<BF16, EPI, TP, TQ, 256, 256, 2, 4><<<grid, 512, 0, stream>>>(g);
    else if (shape == 1) product_kernel<BF16, EPI, TP, TQ, 128, 128, 2, 2><<<grid, 256, 0, stream>>>(g);
    else product_kernel<BF16, EPI, TP, TQ, 128, 32, 4, 1><<<grid, 256, 0, stream>>>(g);
}

void set_tiles(Product &g, int shape, int splits) {
    g.tiles_p = (int)ceil_div(g.np, kTiles[shape].p);
    g.tiles_q = (int)ceil_div(g.nq, kTiles[shape].q);
    g.splits = splits;
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
    rows_kernel<<<1, 1024, 0, stream>>>(a, sums, map, target);
    if (a.count > 0) idle_rows_kernel<<<(unsigned)ceil_div(a.count, 4), 256, 0, stream>>>(a, losses);
    const void *table = a.table;
    if (p.pack_table) {
        pack_kernel<BF16><<<(unsigned)a.vocab, 256, 0, stream>>>(a.table, a.vocab, a.width, nullptr, nullptr, 0,
                                                                 w + p.table_off, a.vocab, p.width_p);
        table = w + p.table_off;
    }
    for (int64_t k = 0; k < p.pieces; ++k) {
        const int64_t first = k * p.piece;
        pack_kernel<BF16><<<(unsigned)p.piece_p, 256, 0, stream>>>(a.hidden, p.piece, a.width, map, sums, first,
                                                                   w + p.hidden_off, p.piece_p, p.width_p);
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
        set_tiles(g, p.tile_logits, 1);
        start_product<BF16, kLogits, false, false>(g, p.tile_logits, stream);
        softmax_kernel<<<(unsigned)ceil_div(p.piece, 4), 256, 0, stream>>>(a, sums, map, first, p.piece, stat,
                                                                           p.subtiles, rows, losses);
        if (!grads) continue;
        gradient_kernel<BF16><<<dim3((unsigned)ceil_div(p.vocab_p * es, 256 * 16), (unsigned)p.piece_p), 256, 0, stream>>>(
            a, sums, target, first, p.piece, stat, p.subtiles, p.sub, rows, w + p.e_off, p.vocab_p);
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
            set_tiles(h, p.tile_hidden, p.splits);
            if (p.splits > 1) {
                h.f32 = reinterpret_cast<float *>(w + p.split_off);
                h.f32_split = p.piece * a.width;
                start_product<BF16, kF32, true, false>(h, p.tile_hidden, stream);
            } else {
                h.map = map;
                h.out = a.grad_hidden;
                h.f32 = static_cast<float *>(a.grad_hidden);
                start_product<BF16, BF16 ? kBf16 : kF32, true, false>(h, p.tile_hidden, stream);
            }
            if (p.splits > 1)
                join_kernel<BF16><<<(unsigned)p.piece, 256, 0, stream>>>(a, sums, map, first, p.piece, h.f32, p.splits,
                                                                         h.f32_split);
        }
        if (a.grad_table) {
            Product t = {};
            t.sums = sums;
            t.first = first;
            t.piece = p.piece;
            t.p = w + p.hidden_off;
            t.ldp = p.width_p * es;
            t.kp = p.piece_p;
            t.np = a.width;
            t.q = w + p.e_off;
            t.ldq = p.vocab_p * es;
            t.nq = a.vocab;
            t.piece_is_k = true;
            t.ldo = a.width;
            const bool last = k + 1 == p.pieces;
            float *gw = a.table_grad_bf16 ? reinterpret_cast<float *>(w + p.gw_off) : static_cast<float *>(a.grad_table);
            set_tiles(t, p.tile_table, 1);
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
    loss_kernel<<<1, 1024, 0, stream>>>(a, sums, map, losses);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_head(const HeadArgs &a, const HeadPlan &p, hipStream_t stream) {
    return a.bf16 ? head<true>(a, p, stream) : head<false>(a, p, stream);
}

}  // namespace zk
