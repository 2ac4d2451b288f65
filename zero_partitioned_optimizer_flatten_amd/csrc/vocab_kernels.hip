// Embedding lookup, its gradient by sorted tokens, and dropout, for gfx950.
//
// Arithmetic is binary32; every output is rounded once (nearest, ties to
// even). No floating-point atomics: the same call gives the same bits.
#include <type_traits>

#include "vocab_internal.h"

namespace zk {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;           // elements of one vector, one Philox block

// ------------------------------------------------------------ elements

// To bf16, nearest, ties to even, NaN kept: two to an instruction.
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    typedef __attribute__((ext_vector_type(2))) float f32x2_t;
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
    const f32x2_t x = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2_t));
}

// V elements at any alignment of their type, of which `left` exist.
template <bool BF16, int V = kVec> struct Raw {
    static constexpr int kWords = V * (BF16 ? 2 : 4) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const void *base, int64_t at, int64_t left) {
        if (left >= V) {
            __builtin_memcpy(w, static_cast<const char *>(base) + at * (BF16 ? 2 : 4), sizeof w);
        } else if constexpr (BF16) {
            const uint16_t *p = static_cast<const uint16_t *>(base) + at;
#pragma unroll
            for (int k = 0; k < kWords; ++k)
                w[k] = (2 * k < left ? p[2 * k] : 0u) | (2 * k + 1 < left ? (uint32_t)p[2 * k + 1] << 16 : 0u);
        } else {
            const uint32_t *p = static_cast<const uint32_t *>(base) + at;
#pragma unroll
            for (int k = 0; k < kWords; ++k) w[k] = k < left ? p[k] : 0u;
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < kWords; ++k) w[k] = 0u;
    }
    __device__ __forceinline__ void get(float *v) const {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if constexpr (BF16) v[k] = __uint_as_float(k % 2 ? w[k / 2] & 0xFFFF0000u : w[k / 2] << 16);
            else v[k] = __uint_as_float(w[k]);
        }
    }
};

// NT: past the caches.
template <bool BF16, int V = kVec, bool NT = false>
__device__ __forceinline__ void store(void *base, int64_t at, int64_t left, const float *v) {
    using T = std::conditional_t<BF16, uint16_t, float>;
    T *p = static_cast<T *>(base) + at, h[V];
    if constexpr (BF16) {
        uint32_t w[V / 2];
#pragma unroll
        for (int k = 0; k < V / 2; ++k) w[k] = narrow2(v[2 * k], v[2 * k + 1]);
        __builtin_memcpy(h, w, sizeof h);
    } else {
        __builtin_memcpy(h, v, sizeof h);
    }
    if (left >= V) {
        if constexpr (NT) {
            static_assert(sizeof h == 16, "one vector");
            typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4;
            __builtin_nontemporal_store(__builtin_bit_cast(u32x4, h), reinterpret_cast<u32x4 *>(p));
        } else {
            __builtin_memcpy(p, h, sizeof h);
        }
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < left) p[k] = h[k];
    }
}

// ------------------------------------------------------------- dropout
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011): 128 bits for each counter (block, offset), used as
// eight 16-bit numbers. With 16 bits an element instead of 32 the ten rounds'
// 20 wide products, which issue at a quarter of the rate, serve twice as many
// elements; p is then a multiple of 2^-16, and the scale is the inverse of the
// share that this p keeps, so the expectation stays exact.

struct Bits8 {
    uint32_t w[4];                // element k: the k-th 16 bits
};

__device__ __forceinline__ Bits8 philox(uint64_t block, uint64_t offset, uint32_t k0, uint32_t k1) {
    uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32);
    uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return {{c0, c1, c2, c3}};
}

__device__ __forceinline__ uint64_t drop_offset(const Drop &d) {
    return d.offset + (d.limit && d.counter ? *d.counter : 0);
}

// v[k] = keep(first + k) ? v[k] * scale : 0 for V elements, four or eight, from
// any place; ALIGNED: from a multiple of V. A dropped element is a selected zero,
// so NaN and infinity there vanish.
template <bool ALIGNED, int V = kVec>
__device__ __forceinline__ void drop(const Drop &d, uint64_t offset, uint64_t first, float *v) {
    const Bits8 x = philox(first / kVec, offset, d.key0, d.key1);
    const int s = (int)(first % kVec);
    if (ALIGNED || s % V == 0) {
        const uint32_t *w = x.w;
        uint32_t part[V / 2];
#pragma unroll
        for (int k = 0; k < V / 2; ++k) part[k] = V == kVec || s == 0 ? w[k] : w[(k + kVec / 2 - V / 2) % 4];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const uint32_t u = (part[k / 2] >> (16 * (k % 2))) & 0xFFFFu;
            v[k] = u >= d.limit ? v[k] * d.scale : 0.0f;
        }
    } else {
        const Bits8 y = philox(first / kVec + 1, offset, d.key0, d.key1);
        uint32_t keep = 0;
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            keep |= (uint32_t)(((x.w[k / 2] >> (16 * (k % 2))) & 0xFFFFu) >= d.limit) << k;
            keep |= (uint32_t)(((y.w[k / 2] >> (16 * (k % 2))) & 0xFFFFu) >= d.limit) << (k + kVec);
        }
        keep >>= s;
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = (keep >> k) & 1u ? v[k] * d.scale : 0.0f;
    }
}

// 16 bytes of output to a lane. Bound by memory: 2^28 bf16 elements take 168 us
// (1.07 GB, 6.4 TB/s; the random numbers' 20 wide products for 8 elements hide
// behind it). Two and four vectors to a thread, all asked for before the first is
// used, took 178 and 180 us: waves enough are under way without.
template <bool BF16, bool ADD, bool NT>
__global__ void __launch_bounds__(kThreads) dropout_kernel(DropoutArgs a) {
    constexpr int V = BF16 ? 8 : 4;
    const int64_t at = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * V, left = a.count - at;
    if (left <= 0) return;
    Raw<BF16, V> x, r;
    float v[V], w[V];
    x.load(a.x, at, left);
    if (ADD) r.load(a.add, at, left);
    x.get(v);
    drop<true, V>(a.drop, drop_offset(a.drop), (uint64_t)at, v);
    if (ADD) {
        r.get(w);
#pragma unroll
        for (int c = 0; c < V; ++c) v[c] += w[c];
    }
    store<BF16, V, NT>(a.out, at, left, v);
}

// -------------------------------------------------------------- lookup

__device__ __forceinline__ int64_t load_id(const void *ids, bool wide, int64_t i) {
    return wide ? static_cast<const int64_t *>(ids)[i] : (int64_t) static_cast<const int32_t *>(ids)[i];
}

// 16 bytes of an output row to a lane. Bound by memory: 20480 rows of 4096 bf16
// take 47.4 us (2 x 168 MB, many of the rows read from caches: 7.1 TB/s); with four
// vectors to a thread 50.0.
template <bool TBF, bool OBF, bool POS, bool DROP, bool ALIGNED, bool NT>
__global__ void __launch_bounds__(kThreads) embed_kernel(EmbedArgs a, uint32_t per_row) {
    constexpr int V = OBF ? 8 : 4;
    const uint32_t unit = blockIdx.x * kThreads + threadIdx.x;      // below 2^32
    const uint32_t row = unit / per_row;
    if (row >= a.count) return;
    const int64_t col = (int64_t)(unit - row * per_row) * V, left = a.width - col;
    const int64_t id = load_id(a.ids, a.wide_ids, row);
    const int64_t pos = POS ? load_id(a.pos_ids, a.wide_ids, row) : -1;
    Raw<TBF, V> x, r;
    if ((uint64_t)id < (uint64_t)a.rows) x.load(a.table, id * a.width + col, left);
    else x.clear();
    if (POS) {
        if ((uint64_t)pos < (uint64_t)a.pos_rows) r.load(a.pos_table, pos * a.width + col, left);
        else r.clear();
    }
    float v[V], w[V];
    x.get(v);
#pragma unroll
    for (int c = 0; c < V; ++c) v[c] *= a.scale;
    if (POS) {
        r.get(w);
#pragma unroll
        for (int c = 0; c < V; ++c) v[c] += w[c];
    }
    const int64_t at = (int64_t)row * a.width + col;
    if (DROP) drop<ALIGNED, V>(a.drop, drop_offset(a.drop), (uint64_t)at, v);
    store<OBF, V, NT>(a.out, at, left, v);
}

// ------------------------------------------- gradient: tokens, sorted
// The tokens are grouped by id in one launch with no traffic between its
// workgroups. Workgroup g owns the ids that are g modulo the workgroup count
// (a power of two; neighbouring ids, which frequencies go by, end up in
// different ones) and reads every token: it counts its own ids, and how many
// tokens belong to the workgroups before it, which is where its share of the
// sorted list begins. A second reading places its tokens, each wave its own
// stretch of the batch in order, so equal ids keep the order they came in and
// their sum is always added up the same way. When the gradient is written and
// not added to, the rows of ids that no token names are set to zero here.
//
// Up to 8192 tokens a wave's ids stay in its registers and the second reading is left
// out. Those take 9 us, of which a workgroup's own 6.7 (text's tokens, 50257 rows):
// clearing its counts 0.5, reading and counting 1.6, the waves' sums 1.2, begins and
// places 1.2, placing 2.2. Beyond, counting and placing grow with the tokens of a wave
// (131072: 23 and 34 of 59), and where most tokens are of one id their additions to one
// number queue up (8192 of one id 12 us in its workgroup, 131072 150). Written and not
// added to, the zeros follow: 16384 tokens, 32000 rows of 4096 bf16 take 51 us.

__device__ __forceinline__ void zero_row(char *p, int64_t bytes, int lane) {
    // 2-byte elements up to a 16-byte line, whole vectors, the rest
    int64_t head = (16 - ((uintptr_t)p & 15)) & 15;
    if (head > bytes) head = bytes;
    for (int64_t k = 2 * lane; k < head; k += 128) *reinterpret_cast<uint16_t *>(p + k) = 0;
    const int64_t vecs = (bytes - head) / 16;
    typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
    const u32x4 z = {0, 0, 0, 0};
    for (int64_t k = lane; k < vecs; k += 64) __builtin_nontemporal_store(z, reinterpret_cast<u32x4 *>(p + head + 16 * k));
    for (int64_t k = head + 16 * vecs + 2 * lane; k < bytes; k += 128)
        *reinterpret_cast<uint16_t *>(p + k) = 0;
}

// Ids a lane has under way.
constexpr int kSortBatch = 8;

__global__ void __launch_bounds__(64 * kSortWaves)
sort_kernel(EmbedGradArgs a, int log2_groups, int per_group, SortedToken *sorted, int32_t *total) {
    extern __shared__ int32_t counts[];            // [kSortWaves][per_group], then places
    __shared__ int32_t before[kSortWaves], sums[kSortWaves];
    int32_t *begin = counts + kSortWaves * per_group, *end = begin + per_group;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const uint32_t group = blockIdx.x, mask = (1u << log2_groups) - 1;
    for (int k = threadIdx.x; k < kSortWaves * per_group; k += 64 * kSortWaves) counts[k] = 0;
    __syncthreads();
    const int64_t stretch = (a.count + 64 * kSortWaves - 1) / (64 * kSortWaves) * 64;
    const int64_t first = stretch * wave;
    const int64_t last = first + stretch < a.count ? first + stretch : a.count;
    int32_t *mine = counts + wave * per_group;
    int32_t lower = 0, all = 0;
    int64_t ids[kSortBatch];
    // kSortBatch * 64 ids from i0, -1 for those outside the table or the stretch
    auto load = [&](int64_t i0) {
#pragma unroll
        for (int k = 0; k < kSortBatch; ++k) {
            const int64_t i = i0 + 64 * k + lane;
            ids[k] = i < last ? load_id(a.ids, a.wide_ids, i) : -1;
        }
#pragma unroll
        for (int k = 0; k < kSortBatch; ++k)
            if ((uint64_t)ids[k] >= (uint64_t)a.rows) ids[k] = -1;
    };
    for (int64_t i0 = first; i0 < last; i0 += 64 * kSortBatch) {
        load(i0);
#pragma unroll
        for (int k = 0; k < kSortBatch; ++k) {
            if (ids[k] < 0) continue;
            const uint32_t g = (uint32_t)ids[k] & mask;
            lower += g < group;
            ++all;
            if (g == group) atomicAdd(&mine[(uint32_t)ids[k] >> log2_groups], 1);
        }
    }
    for (int s = 32; s; s /= 2) {
        lower += __shfl_xor(lower, s);
        all += __shfl_xor(all, s);
    }
    if (lane == 0) before[wave] = lower, sums[wave] = all;
    __syncthreads();
    int32_t base = 0;
    all = 0;
    for (int w = 0; w < kSortWaves; ++w) {
        base += before[w];
        all += sums[w];
    }
    if (group == 0 && threadIdx.x == 0) *total = all;
    __syncthreads();
    // one id to a thread (per_group <= kSortIds): an exclusive sum over the ids
    int32_t own = 0;
    if ((int)threadIdx.x < per_group)
        for (int w = 0; w < kSortWaves; ++w) own += counts[w * per_group + threadIdx.x];
    int32_t upto = own;
    for (int s = 1; s < 64; s *= 2) {
        const int32_t x = __shfl_up(upto, s);
        if (lane >= s) upto += x;
    }
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    for (int w = 0; w < wave; ++w) base += sums[w];
    if ((int)threadIdx.x < per_group) {
        int32_t at = base + upto - own;
        begin[threadIdx.x] = at;
        end[threadIdx.x] = at + own;
        for (int w = 0; w < kSortWaves; ++w) {
            const int32_t c = counts[w * per_group + threadIdx.x];
            counts[w * per_group + threadIdx.x] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int64_t i0 = first; i0 < last; i0 += 64 * kSortBatch) {
        if (stretch > 64 * kSortBatch) load(i0);    // else they are still there
#pragma unroll
        for (int b = 0; b < kSortBatch; ++b) {
            const bool here = ids[b] >= 0 && ((uint32_t)ids[b] & mask) == group;
            const int32_t k = here ? (int32_t)((uint32_t)ids[b] >> log2_groups) : -1;
            uint64_t todo = __ballot(here);
            while (todo) {                           // the ids among these 64, one by one
                const int leader = __builtin_ctzll(todo);
                const uint64_t same = __ballot(k == __shfl(k, leader));
                int32_t at = 0;
                if (lane == leader) at = atomicAdd(&mine[k], (int32_t)__popcll(same));
                at = __shfl(at, leader) + __popcll(same & ((1ull << lane) - 1));
                if ((same >> lane) & 1)
                    sorted[at] = {(int32_t)ids[b], (int32_t)(i0 + 64 * b + lane), begin[k], end[k]};
                todo &= ~same;
            }
        }
    }
    if (a.accumulate) return;
    const int64_t row_bytes = a.width * (a.out_bf16 ? 2 : 4);
    for (int k = wave; k < per_group; k += kSortWaves) {
        const int64_t id = ((int64_t)k << log2_groups) + group;
        if (id < a.rows && begin[k] == end[k])
            zero_row(static_cast<char *>(a.out) + id * row_bytes, row_bytes, lane);
    }
}

// ------------------------------------------- gradient: runs added up
// A wave adds up `span` sorted tokens, 512 columns of them, in order. A run of
// equal ids inside the span is one row of the gradient and written at once. Of
// a run that goes over the span's end or came in over its start the wave
// leaves a partial row: slot 2s where it came in, else slot 2s + 1. The joining
// kernel adds a run's partial rows in the order of the spans. So the work is
// even whatever the tokens are, one padding token a million times included. Bound by
// memory: 16384 rows of 4096 bf16 (134 MB), a third of them of one id, take 42 us,
// and 7 the joining. The sums are in binary32, the partial rows too; a row is rounded once, when it is written.

// Rows a lane has under way.
constexpr int kSpanBatch = 8;

// A whole row of the gradient from its sum; `old` what it holds, to be added to.
template <bool OBF>
__device__ __forceinline__ void write_row(const EmbedGradArgs &a, int32_t id, int64_t col,
                                          const float *sum, const Raw<OBF> &old) {
    const int64_t left = a.width - col;
    if (left <= 0) return;
    float v[kVec], o[kVec];
    old.get(o);
#pragma unroll
    for (int k = 0; k < kVec; ++k) v[k] = a.accumulate ? sum[k] * a.scale + o[k] : sum[k] * a.scale;
    store<OBF>(a.out, (int64_t)id * a.width + col, left, v);
}

template <bool GBF, bool OBF, bool DROP, bool ALIGNED>
__global__ void __launch_bounds__(kThreads)
span_kernel(EmbedGradArgs a, const SortedToken *sorted, const int32_t *total, int span,
            int col_chunks, float *partial, int64_t pitch) {
    const int unit = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + threadIdx.x / 64);
    const int lane = threadIdx.x % 64;
    const int s = __builtin_amdgcn_readfirstlane((uint32_t)unit / (uint32_t)col_chunks);
    const int64_t col = (int64_t)(unit - s * col_chunks) * kSpanCols + lane * kVec;
    const int n = __builtin_amdgcn_readfirstlane(*total);
    int64_t lo = (int64_t)s * span;
    if (lo >= n) return;
    const int64_t hi = lo + span < n ? lo + span : n;
    const int64_t left = a.width - col;
    const uint64_t offset = DROP ? drop_offset(a.drop) : 0;
    float sum[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) sum[k] = 0.0f;
    for (int64_t i0 = lo; i0 < hi; i0 += 64) {
        const int m = (int)(hi - i0 < 64 ? hi - i0 : 64);
        SortedToken t = {0, 0, 0, 0};
        if (lane < m) t = sorted[i0 + lane];
        // whether a token ends a run that is all in the span
        const bool ends = lane < m && t.end == i0 + lane + 1 && t.begin >= lo;
        const uint64_t whole = __ballot(ends);
        for (int k0 = 0; k0 < m; k0 += kSpanBatch) {
            Raw<GBF> raw[kSpanBatch];
            Raw<OBF> old[kSpanBatch];
#pragma unroll
            for (int k = 0; k < kSpanBatch; ++k) {
                const int row = __builtin_amdgcn_readlane(t.row, (k0 + k) % 64);   // 0 behind the last
                if (left > 0) raw[k].load(a.grad_out, (int64_t)row * a.width + col, left);
            }
            if (a.accumulate)
#pragma unroll
                for (int k = 0; k < kSpanBatch; ++k) {
                    const int id = __builtin_amdgcn_readlane(t.id, (k0 + k) % 64);
                    if (left > 0 && whole >> (k0 + k) % 64 & 1) old[k].load(a.out, (int64_t)id * a.width + col, left);
                }
#pragma unroll
            for (int k = 0; k < kSpanBatch; ++k) {
                if (k0 + k >= m) break;
                const int row = __builtin_amdgcn_readlane(t.row, k0 + k), end = __builtin_amdgcn_readlane(t.end, k0 + k);
                if (left > 0) {
                    float v[kVec];
                    raw[k].get(v);
                    if (DROP) drop<ALIGNED>(a.drop, offset, (uint64_t)row * a.width + col, v);
#pragma unroll
                    for (int c = 0; c < kVec; ++c) sum[c] += v[c];
                }
                const int64_t i = i0 + k0 + k;
                if (i + 1 == end || i + 1 == hi) {
                    const int begin = __builtin_amdgcn_readlane(t.begin, k0 + k);
                    if (begin >= lo && end <= hi) {
                        write_row<OBF>(a, __builtin_amdgcn_readlane(t.id, k0 + k), col, sum, old[k]);
                    } else if (left > 0) {
                        float *p = partial + (2 * (int64_t)s + (begin >= lo)) * pitch + col;
                        __builtin_memcpy(__builtin_assume_aligned(p, 16), sum, sizeof sum);
                    }
#pragma unroll
                    for (int c = 0; c < kVec; ++c) sum[c] = 0.0f;
                }
            }
        }
    }
}

// For few tokens, where a joining kernel would take as long as the sums: workgroup
// (token, columns) adds up the run that begins at the token. Its rows are dealt to
// the waves in stretches, joined in order; a short run is the first wave's.
constexpr int kRunWaves = 8;

template <bool GBF, bool OBF, bool DROP>
__global__ void __launch_bounds__(64 * kRunWaves)
run_kernel(EmbedGradArgs a, const SortedToken *sorted, const int32_t *total, int col_chunks) {
    __shared__ __align__(16) float sums[kRunWaves][kSpanCols];
    const int s = __builtin_amdgcn_readfirstlane(blockIdx.x / (uint32_t)col_chunks);
    if (s >= *total) return;                       // the whole workgroup, as below
    const SortedToken t = sorted[s];
    if (t.begin != s) return;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t col = (int64_t)(blockIdx.x - (uint32_t)s * col_chunks) * kSpanCols + lane * kVec, left = a.width - col;
    const int end = __builtin_amdgcn_readfirstlane(t.end), length = end - s;
    const bool split = length > kSpanBatch;
    const int each = split ? (length + kRunWaves - 1) / kRunWaves : length;
    const int lo = s + each * wave, hi = lo + each < end ? lo + each : end;
    const uint64_t offset = DROP ? drop_offset(a.drop) : 0;
    Raw<OBF> old;
    old.clear();
    if (a.accumulate && wave == 0 && left > 0) old.load(a.out, (int64_t)t.id * a.width + col, left);
    float sum[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) sum[k] = 0.0f;
    for (int k0 = lo; k0 < hi; k0 += kSpanBatch) {
        Raw<GBF> raw[kSpanBatch];
        int row[kSpanBatch];
#pragma unroll
        for (int k = 0; k < kSpanBatch; ++k) row[k] = sorted[k0 + k < hi ? k0 + k : hi - 1].row;
#pragma unroll
        for (int k = 0; k < kSpanBatch; ++k)
            if (left > 0) raw[k].load(a.grad_out, (int64_t)row[k] * a.width + col, left);
#pragma unroll
        for (int k = 0; k < kSpanBatch; ++k) {
            if (k0 + k >= hi || left <= 0) break;
            float v[kVec];
            raw[k].get(v);
            if (DROP) drop<false>(a.drop, offset, (uint64_t)row[k] * a.width + col, v);
#pragma unroll
            for (int c = 0; c < kVec; ++c) sum[c] += v[c];
        }
    }
    if (split) {
        __builtin_memcpy(&sums[wave][lane * kVec], sum, sizeof sum);
        __syncthreads();
    }
    if (wave != 0) return;
    if (split)
        for (int w = 1; w < kRunWaves; ++w)
#pragma unroll
            for (int k = 0; k < kVec; ++k) sum[k] += sums[w][lane * kVec + k];
    write_row<OBF>(a, t.id, col, sum, old);
}

// Workgroup (span, columns): the run that begins in the span and goes over its
// end. Its spans are dealt to the workgroup's waves in stretches, joined in order.
constexpr int kJoinWaves = 4;

template <bool OBF>
__global__ void __launch_bounds__(64 * kJoinWaves)
join_kernel(EmbedGradArgs a, const SortedToken *sorted, const int32_t *total, int span,
            int col_chunks, const float *partial, int64_t pitch) {
    __shared__ __align__(16) float sums[kJoinWaves][kSpanCols];
    const int64_t s = blockIdx.x / col_chunks;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int64_t col = (int64_t)(blockIdx.x % col_chunks) * kSpanCols + lane * kVec;
    const int32_t n = *total;
    const int64_t hi = (s + 1) * span;
    if (hi >= n) return;                           // the whole workgroup
    const SortedToken t = sorted[hi - 1];
    if (t.end <= hi || t.begin < hi - span) return;
    const int64_t last = (t.end - 1) / span;       // the run's last span
    const int64_t more = last - s;                 // slots 2(s+1), 2(s+2), ...
    const int64_t each = (more + kJoinWaves - 1) / kJoinWaves;
    const int64_t b = s + 1 + each * wave, e = b + each < last + 1 ? b + each : last + 1;
    float sum[kVec], v[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) sum[k] = 0.0f;
    if (col < a.width) {
        if (wave == 0) __builtin_memcpy(sum, partial + (2 * s + 1) * pitch + col, sizeof sum);
#pragma unroll 4
        for (int64_t q = b; q < e; ++q) {
            __builtin_memcpy(v, partial + 2 * q * pitch + col, sizeof v);
#pragma unroll
            for (int k = 0; k < kVec; ++k) sum[k] += v[k];
        }
    }
    __builtin_memcpy(&sums[wave][lane * kVec], sum, sizeof sum);
    __syncthreads();
    if (wave != 0) return;
    for (int w = 1; w < kJoinWaves; ++w)
#pragma unroll
        for (int k = 0; k < kVec; ++k) sum[k] += sums[w][lane * kVec + k];
    Raw<OBF> old;
    if (a.accumulate && col < a.width) old.load(a.out, (int64_t)t.id * a.width + col, a.width - col);
    write_row<OBF>(a, t.id, col, sum, old);
}

static_assert(kSpanCols == 64 * kVec, "a vector to a lane");

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// An output of more bytes is stored past the caches, which then keep what is read
// (2^24 bf16 dropped 11.7 us for 14.2, 20480 rows of 4096 looked up 47.4 for 57.4);
// a smaller one (2^22: 4.9 either way) stays where its reader finds it.
constexpr int64_t kCachedBytes = (int64_t)8 << 20;

template <bool TBF, bool OBF, bool POS, bool DROP, bool ALIGNED>
void start_embed(const EmbedArgs &a, hipStream_t stream) {
    const uint32_t per_row = (uint32_t)ceil_div(a.width, OBF ? 8 : 4);
    const int64_t units = a.count * per_row;
    const dim3 grid((unsigned)ceil_div(units, kThreads));
    if (16 * units <= kCachedBytes) embed_kernel<TBF, OBF, POS, DROP, ALIGNED, false><<<grid, kThreads, 0, stream>>>(a, per_row);
    else embed_kernel<TBF, OBF, POS, DROP, ALIGNED, true><<<grid, kThreads, 0, stream>>>(a, per_row);
}

template <bool TBF, bool OBF, bool POS>
void start_embed(const EmbedArgs &a, hipStream_t stream) {
    if (a.drop.limit == 0) start_embed<TBF, OBF, POS, false, true>(a, stream);
    else if (a.width % (OBF ? 8 : 4) == 0) start_embed<TBF, OBF, POS, true, true>(a, stream);
    else start_embed<TBF, OBF, POS, true, false>(a, stream);
}

template <bool BF16, bool ADD>
void start_dropout(const DropoutArgs &a, hipStream_t stream) {
    const int64_t units = ceil_div(a.count, BF16 ? 8 : 4);
    const dim3 grid((unsigned)ceil_div(units, kThreads));
    if (16 * units <= kCachedBytes) dropout_kernel<BF16, ADD, false><<<grid, kThreads, 0, stream>>>(a);
    else dropout_kernel<BF16, ADD, true><<<grid, kThreads, 0, stream>>>(a);
}

template <bool GBF, bool OBF>
void start_spans(const EmbedGradArgs &a, const EmbedGradPlan &p, const SortedToken *sorted,
                 const int32_t *total, float *partial, hipStream_t stream) {
    const int chunks = (int)ceil_div(a.width, kSpanCols);
    const int64_t pitch = (int64_t)chunks * kSpanCols;
    if (p.span == 1) {
        const dim3 grid((unsigned)(a.count * chunks));
        if (a.drop.limit == 0) run_kernel<GBF, OBF, false><<<grid, 64 * kRunWaves, 0, stream>>>(a, sorted, total, chunks);
        else run_kernel<GBF, OBF, true><<<grid, 64 * kRunWaves, 0, stream>>>(a, sorted, total, chunks);
        return;
    }
    const dim3 grid((unsigned)ceil_div(p.spans * chunks, kThreads / 64));
    const bool aligned = a.width % kVec == 0;
#define ZERO_SPANS(DROP, ALIGNED)                                      \
    span_kernel<GBF, OBF, DROP, ALIGNED><<<grid, kThreads, 0, stream>>>( \
        a, sorted, total, p.span, chunks, partial, pitch)
    if (a.drop.limit == 0) ZERO_SPANS(false, true);
    else if (aligned) ZERO_SPANS(true, true);
    else ZERO_SPANS(true, false);
#undef ZERO_SPANS
    if (p.spans > 1)
        join_kernel<OBF><<<dim3((unsigned)((p.spans - 1) * chunks)), 64 * kJoinWaves, 0, stream>>>(
            a, sorted, total, p.span, chunks, partial, pitch);
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs &a, hipStream_t stream) {
    if (a.count == 0) return hipSuccess;
    if (a.bf16) {
        if (a.add) start_dropout<true, true>(a, stream);
        else start_dropout<true, false>(a, stream);
    } else {
        if (a.add) start_dropout<false, true>(a, stream);
        else start_dropout<false, false>(a, stream);
    }
    return hipGetLastError();
}

hipError_t launch_embed(const EmbedArgs &a, hipStream_t stream) {
    if (a.count == 0) return hipSuccess;
    if (a.table_bf16) {
        if (a.out_bf16) {
            if (a.pos_ids) start_embed<true, true, true>(a, stream);
            else start_embed<true, true, false>(a, stream);
        } else {
            if (a.pos_ids) start_embed<true, false, true>(a, stream);
            else start_embed<true, false, false>(a, stream);
        }
    } else {
        if (a.out_bf16) {
            if (a.pos_ids) start_embed<false, true, true>(a, stream);
            else start_embed<false, true, false>(a, stream);
        } else {
            if (a.pos_ids) start_embed<false, false, true>(a, stream);
            else start_embed<false, false, false>(a, stream);
        }
    }
    return hipGetLastError();
}

hipError_t launch_embed_grad(const EmbedGradArgs &a, const EmbedGradPlan &p, hipStream_t stream) {
    if (a.count == 0 && a.accumulate) return hipSuccess;
    auto *sorted = reinterpret_cast<SortedToken *>(a.workspace + p.sorted_off);
    auto *total = reinterpret_cast<int32_t *>(a.workspace + p.count_off);
    auto *partial = reinterpret_cast<float *>(a.workspace + p.partial_off);
    const size_t lds = (size_t)(kSortWaves + 2) * p.ids_per_group * sizeof(int32_t);
    sort_kernel<<<dim3(1u << p.sort_groups_log2), 64 * kSortWaves, lds, stream>>>(
        a, p.sort_groups_log2, p.ids_per_group, sorted, total);
    if (a.count > 0) {
        if (a.grad_bf16) {
            if (a.out_bf16) start_spans<true, true>(a, p, sorted, total, partial, stream);
            else start_spans<true, false>(a, p, sorted, total, partial, stream);
        } else {
            if (a.out_bf16) start_spans<false, true>(a, p, sorted, total, partial, stream);
            else start_spans<false, false>(a, p, sorted, total, partial, stream);
        }
    }
    return hipGetLastError();
}

}  // namespace zk
