// gfx950 kernels for AdamW over many tensors at once, with fp32 or 8-bit
// states, and for the sum of squares of the mean gradient it clips by.
//
// Per element, in binary32 unless said otherwise (k: the element's tensor):
//     g   = (g_0 + ... + g_{N-1}) / N              (left fold, rank order)
//     g   = g * f32(min(1, max_norm / (sqrt(S) + 1e-6)))   with clipping
//     lr_k = lr * factor_k;  keep_k = 1 - lr_k * decay_k
//   32-bit states
//     m = fma(g, 1-b1, m*b1);  v = fma((1-b2)*g, g, v*b2)
//     p = p * keep_k - (lr_k * (m / bc1)) / (sqrt(v / bc2) + eps)
//   8-bit states: m and r = sqrt(v) are held as e4m3 codes, 32 elements to a
//   power-of-two scale
//     m = fma(g, 1-b1, m*b1);  v = fma((1-b2)*g, g, (r*r)*b2);  r = sqrt(v)
//     p = p * keep_k - (lr_k / bc1) * (m / (r * (1/sqrt(bc2)) + eps))
// with bc = 1 - b^t. The 32-bit step without decay and clipping is bit for
// bit the per-parameter step of zero_kernels.hip.
//
// All of it is bound by HBM: 0.6 to 1.5 operations per byte by these formulas.
// The 8-bit step with its roots, codes and noise takes about 50 vector
// instructions per element, which keep the vector units 62% busy; every
// one of them counts there.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_internal.h"

namespace zk {

namespace {

constexpr int kWave = 64;
constexpr int kQuad = 4;                         // elements per lane and load
constexpr int kSplit = 2;                        // quads of a lane
constexpr int kWaveElems = kSplit * kQuad * kWave;   // a wave's part of a piece
constexpr int kPieceWaves = kAdamwPiece / kWaveElems;

// Dynamic LDS that a workgroup reserves and does not touch, to set how many
// share a compute unit (160 KiB each).
// 32-bit states, one-wave workgroups, 7 per unit: 3.94 ms on the Llama-7B list
// (rank of 8, reduced fp32 gradients) and 537 us on GPT-2 small whole, against
// 3.97 and 541 at 8, 3.98 and 550 at 10, 4.19 and 544 at 14, 3.96 and 541 at 6
// (one state, all variants in turn).
constexpr unsigned kLds32 = 22528;
// 8-bit states, one piece per workgroup (so that each 128-byte line of scales
// is one workgroup's), 3 per unit: 2.16 ms on the same list wherever its
// buffers came to lie; 4 per unit took 2.12 or 2.25 by their placement, 6 took
// 2.15 or 2.31, 2 took 2.49, uncapped 2.14 to 2.28.
constexpr unsigned kLds8 = 53248;
// Cache policies of buffer instructions (gfx950: nt = 2, sc1 = 16). Loads and
// stores stream (nt): what a step touches does not outlive the forward and
// backward pass that follows it in the Infinity Cache. Default-policy stores
// ran at 4.60 ms where nt ones took 4.05 (32 bits, Llama-7B) and 2.58 where
// these took 2.38 (8 bits).
constexpr int kPolDefault = 0, kPolNT = 2;
// A state of more than half the 256 MB Infinity Cache (11M elements with 32
// bits, 22M with 8) is stored at device scope as well (nt sc1). Device scope
// against nt, us, on eight or ten states in turn that leave nothing in a cache:
//   32 bits           4M           8M          12M          20M elements
//   reduced bf16  21.3  21.0   38.1  38.3   55.2  55.6   89.9  91.5
//   reduced fp32  24.3  23.9   43.6  43.2   63.9  63.4  103.4 103.5
//   4 of bf16     25.7  26.1   47.4  48.0   67.7  69.5  108.9 110.3
//   8 of bf16     31.0  30.7   56.4  56.7   82.6  83.0  133.6 134.3
//   8 bits           12M          24M          36M          56M elements
//   reduced bf16  34.9  34.1   64.6  64.1   94.7  95.0  144.3 145.7
//   reduced fp32  41.7  41.4   79.4  79.4  118.2 118.6  184.0 184.1
//   4 of bf16     45.1  45.6   85.1  86.3  126.3 128.1  195.7 197.8
//   8 of bf16     60.6  60.5  116.9 117.2  174.0 173.7  272.0 271.5
// and 3.92-3.95 ms against 3.96-4.05 and 2.09 against 2.12 (Llama-7B).
constexpr int kPolDevice = 18;

template <int V> struct Const { static constexpr int value = V; };

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __amdgpu_buffer_rsrc_t span_t;

// A descriptor over `nbytes` at a wave-uniform address, for instructions
// that take a lane's byte offset into it and a cache policy.
__device__ __forceinline__ span_t span_of(const void *base, int nbytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, nbytes,
                                             0x00020000);
}

__device__ __forceinline__ float widen_bf16(uint32_t bits16) {
    return __uint_as_float(bits16 << 16);
}

// Two values to bf16, nearest, ties to even, NaN kept (one instruction).
__device__ __forceinline__ uint32_t round_bf16x2(float lo, float hi) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    const f32x2_t x = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2_t));
}

template <bool B>
__device__ __forceinline__ float elem(const void *base, int64_t i) {
    return B ? widen_bf16(static_cast<const uint16_t *>(base)[i])
             : static_cast<const float *>(base)[i];
}

// Four elements as loaded: 8 bytes of bf16 or 16 of fp32.
template <bool B> struct RawQuad;
template <> struct RawQuad<true> { u32x2_t w; };
template <> struct RawQuad<false> { u32x4_t w; };

__device__ __forceinline__ void widen(const RawQuad<true> &r, float (&x)[kQuad]) {
    x[0] = widen_bf16(r.w.x & 0xFFFFu);
    x[1] = __uint_as_float(r.w.x & 0xFFFF0000u);
    x[2] = widen_bf16(r.w.y & 0xFFFFu);
    x[3] = __uint_as_float(r.w.y & 0xFFFF0000u);
}
__device__ __forceinline__ void widen(const RawQuad<false> &r, float (&x)[kQuad]) {
    x[0] = __uint_as_float(r.w.x);
    x[1] = __uint_as_float(r.w.y);
    x[2] = __uint_as_float(r.w.z);
    x[3] = __uint_as_float(r.w.w);
}

template <bool B>
__device__ __forceinline__ RawQuad<B> narrow(const float (&x)[kQuad]) {
    RawQuad<B> r;
    if constexpr (B) {
        r.w.x = round_bf16x2(x[0], x[1]);
        r.w.y = round_bf16x2(x[2], x[3]);
    } else {
        r.w = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
               __float_as_uint(x[3])};
    }
    return r;
}

// A whole quad `off` elements into a wave's part of a caller's buffer, which
// starts at `base`. AL: the part is aligned for the instruction's width, and
// goes through a buffer instruction with its policy; otherwise through a
// load or store at the element's own alignment.
template <bool B, bool AL, int POL>
__device__ __forceinline__ RawQuad<B> load_raw(const char *base, int off) {
    constexpr int es = B ? 2 : 4;
    RawQuad<B> r;
    if constexpr (AL) {
        const span_t sp = span_of(base, kAdamwPiece * es);
        if constexpr (B) r.w = __builtin_amdgcn_raw_buffer_load_b64(sp, off * es, 0, POL);
        else r.w = __builtin_amdgcn_raw_buffer_load_b128(sp, off * es, 0, POL);
    } else {
        __builtin_memcpy(&r, base + off * es, sizeof r);
    }
    return r;
}

template <bool B, bool AL, int POL>
__device__ __forceinline__ void store_raw(char *base, int off, const RawQuad<B> &r) {
    constexpr int es = B ? 2 : 4;
    if constexpr (AL) {
        const span_t sp = span_of(base, kWaveElems * es);
        if constexpr (B) __builtin_amdgcn_raw_buffer_store_b64(r.w, sp, off * es, 0, POL);
        else __builtin_amdgcn_raw_buffer_store_b128(r.w, sp, off * es, 0, POL);
    } else {
        __builtin_memcpy(base + off * es, &r, sizeof r);
    }
}

template <int POL>
__device__ __forceinline__ void load_f4(span_t sp, int off, float (&x)[kQuad]) {
    RawQuad<false> r;
    r.w = __builtin_amdgcn_raw_buffer_load_b128(sp, off * 4, 0, POL);
    widen(r, x);
}
template <int POL>
__device__ __forceinline__ void store_f4(span_t sp, int off, const float (&x)[kQuad]) {
    __builtin_amdgcn_raw_buffer_store_b128(narrow<false>(x).w, sp, off * 4, 0, POL);
}

// The first `left` values of a quad at a tensor's end.
template <bool B>
__device__ __forceinline__ void store_quad(void *base, int64_t i, int64_t left,
                                           const float (&x)[kQuad]) {
    if (left >= kQuad) {
        const RawQuad<B> r = narrow<B>(x);
        __builtin_memcpy(static_cast<char *>(base) + i * (B ? 2 : 4), &r, sizeof r);
    } else {
#pragma unroll
        for (int e = 0; e < kQuad; ++e) {
            if (e < left) {
                if (B) static_cast<uint16_t *>(base)[i + e] = (uint16_t)round_bf16x2(x[e], 0.0f);
                else static_cast<float *>(base)[i + e] = x[e];
            }
        }
    }
}

// What a launch only reads, at addresses that are uniform over a wave, goes
// through the constant address space: scalar loads, and values that the
// compiler knows to be uniform (a descriptor over a pointer it does not know
// to be uniform costs a loop around every access).
#define ZK_CONSTANT __attribute__((address_space(4)))
typedef const ZK_CONSTANT AdamwTensor Tensor;
typedef const ZK_CONSTANT AdamwGroup Group;

template <class T>
__device__ __forceinline__ const ZK_CONSTANT T *constant(const T *p) {
    return (const ZK_CONSTANT T *)(uintptr_t)p;
}

struct KernelArgs {
    const AdamwTensor *table;
    const AdamwGroup *groups;
    const int32_t *map;
    int n;
    AdamwStateRef st;
    StepScalars sc;
    const StepScalars *sc_dev;
    const DevSchedule *ds;
    uint32_t seed, t;
    const double *sumsq;
    double max_norm;
    int stream_state;
};

// The clip factor; false where the sum of squares is not finite, and then
// the step writes nothing.
__device__ __forceinline__ bool clip_factor(const double *sumsq, double max_norm, float &c) {
    c = 1.0f;
    if (!sumsq) return true;
    const double s = *constant(sumsq);
    if (!(s >= 0.0 && s < __builtin_inf())) return false;
    const double f = max_norm / (__builtin_sqrt(s) + 1e-6);
    if (f < 1.0) c = (float)f;
    return true;
}

// What a wave needs beside its data: uniform over the wave. The scalars that
// depend on the replica count are the binding's, also where the schedule's
// come from the device.
struct Uniform {
    StepScalars sc;
    bool pow2;
    float scale;          // of the sum over the replicas: clip factor, and 1/N where exact
    float lr, keep;
};

template <int NR>
__device__ __forceinline__ bool uniforms(const KernelArgs &a, Group &gr, Uniform &u) {
    float clip;
    if (!clip_factor(a.sumsq, a.max_norm, clip)) return false;
    u.sc = a.sc;
    if (a.sc_dev) {
        const ZK_CONSTANT StepScalars &d = *constant(a.sc_dev);
        u.sc.b1 = d.b1; u.sc.c1 = d.c1; u.sc.b2 = d.b2; u.sc.c2 = d.c2;
        u.sc.lr = d.lr; u.sc.eps = d.eps; u.sc.bc1 = d.bc1; u.sc.bc2 = d.bc2;
    }
    u.pow2 = NR > 0 ? (NR & (NR - 1)) == 0 : a.sc.n_pow2 != 0;
    u.scale = u.pow2 ? a.sc.inv_n * clip : clip;      // a power of two: the same bits
    u.lr = u.sc.lr * gr.factor;
    u.keep = 1.0f - u.lr * gr.decay;
    return true;
}

__device__ __forceinline__ void mean_clip(const Uniform &u, float (&g)[kQuad]) {
    if (!u.pow2) {
#pragma unroll
        for (int e = 0; e < kQuad; ++e) g[e] = g[e] / u.sc.nf;
    }
#pragma unroll
    for (int e = 0; e < kQuad; ++e) g[e] = g[e] * u.scale;
}

// Replicas whose loads are in flight together.
constexpr int kGroup = 8;
template <int NR> constexpr int kGroupOf = NR > 0 && NR < kGroup ? NR : kGroup;

// A lane's quad of replicas q0, q0 + 1, ... (as far as they exist) at a
// tensor's end: `left` elements of it exist, the others are zero. All loads
// of a group are on their way before the first is waited for.
template <int NR, bool GB>
__device__ __forceinline__ void load_last(Tensor &tn, int q0, int n, int64_t i, int64_t left,
                                          float (&x)[kGroupOf<NR>][kQuad]) {
    constexpr int es = GB ? 2 : 4, grp = kGroupOf<NR>;
    if (left >= kQuad) {
        RawQuad<GB> raw[grp];
#pragma unroll
        for (int k = 0; k < grp; ++k)
            if (NR > 0 || q0 + k < n)
                __builtin_memcpy(&raw[k], static_cast<const char *>(tn.grads[q0 + k]) + i * es,
                                 sizeof raw[k]);
#pragma unroll
        for (int k = 0; k < grp; ++k)
            if (NR > 0 || q0 + k < n) widen(raw[k], x[k]);
    } else {
#pragma unroll
        for (int k = 0; k < grp; ++k)
            if (NR > 0 || q0 + k < n) {
#pragma unroll
                for (int e = 0; e < kQuad; ++e)
                    x[k][e] = e < left ? elem<GB>(tn.grads[q0 + k], i + e) : 0.0f;
            }
    }
}

// Where an element has 8 bytes of gradients or more, of several replicas whose
// count is known when compiled, the master values load once the moments are
// done, which need everything else. Late against together with the rest, on
// states that nothing keeps in a cache; us for GPT-2 small's rank 3 of 8 and
// 27.8M elements at odd widths (six states in turn), ms for Llama-7B's rank 0
// of 8; bf16 outputs:
//                       32 bits                                8 bits
//   2 bf16    79.6  77.2   144  138   3.98 3.89     48.9 47.6    90.3  86.3   2.49 2.46
//   2 fp32    86.3  86.4   157  153   4.52 4.57     57.0 57.4   100.7 101.3   2.99 3.09
//   4 bf16    88.8  88.0   161  158   4.44 4.49     57.9 57.8   109.3 105.7   3.05 3.14
//   4 fp32   106.3 106.5   190  191   5.75 5.83     77.7 78.1   138.9 143.0   4.23 4.31
//   8 bf16   108.7 108.8   198  198   5.57 5.74     77.1 77.8   147.2 146.8   4.34 4.44
//   8 fp32   150.4 150.8   272  274   8.21 8.20    124.5 123.1  227.4 227.4   6.83 6.90
// One replica: bf16 75 and 72, 3.82 and 3.65; 45 and 43, 2.24 and 2.13. With a
// count known only at run time the late load loses (five: 4.86 ms against
// 4.68).
template <int NR, bool GB> constexpr bool kLateMaster = NR >= 2 && NR * (GB ? 2 : 4) >= 8;

// How a part of a tensor (512 elements, a wave's) is reached. The last part
// loads all that it needs before it waits, like the others: GPT-2 small, rank
// 3 of 8, eight bf16 replicas, 107.4 us against 110.3 quad by quad with 32-bit
// states, 77.5 against 78.7 with 8-bit ones.
enum Part {
    kWhole,        // all of it exists and is aligned for whole-quad instructions
    kUnaligned,    // all of it exists
    kLast,         // the tensor ends in it
};

// Clears what is behind the tensor's last element. Gradient and moments are
// zero there (every factor of the step is finite); the step is not where eps
// is 0.
__device__ __forceinline__ void clear_behind(Tensor &tn, int64_t i0, int lane,
                                             float (&x)[kSplit][kQuad]) {
#pragma unroll
    for (int h = 0; h < kSplit; ++h)
#pragma unroll
        for (int e = 0; e < kQuad; ++e)
            if (i0 + kQuad * (lane + h * kWave) + e >= tn.numel) x[h][e] = 0.0f;
}

// Mean gradients of a lane's quads in a part (element i0 of the tensor on;
// elements behind the tensor's last are zero). `first` runs once the first
// group's loads are on their way: it issues the state's, works out u, and
// says whether the step takes place.
template <int NR, bool GB, Part PT, class F>
__device__ __forceinline__ bool mean_part(Tensor &tn, int nrep, const Uniform &u, int64_t i0,
                                          int lane, float (&g)[kSplit][kQuad], F &&first) {
    const int n = NR > 0 ? NR : nrep;
    constexpr int es = GB ? 2 : 4, grp = kGroupOf<NR>;
    constexpr bool AL = PT == kWhole;
    if (PT == kLast && !first()) return false;
#pragma unroll 1
    for (int q0 = 0; q0 < n; q0 += grp) {
        float x[kSplit][grp][kQuad];
        if constexpr (PT == kLast) {
#pragma unroll
            for (int h = 0; h < kSplit; ++h) {
                const int64_t i = i0 + kQuad * (lane + h * kWave);
                load_last<NR, GB>(tn, q0, n, i, tn.numel - i, x[h]);
            }
        } else {
            RawQuad<GB> raw[grp][kSplit];
#pragma unroll
            for (int k = 0; k < grp; ++k)
                if (NR > 0 || q0 + k < n) {
                    const char *base = static_cast<const char *>(tn.grads[q0 + k]) + i0 * es;
#pragma unroll
                    for (int h = 0; h < kSplit; ++h)
                        raw[k][h] = load_raw<GB, AL, AL ? kPolNT : kPolDefault>(
                            base, kQuad * (lane + h * kWave));
                }
            if (q0 == 0 && !first()) return false;
#pragma unroll
            for (int k = 0; k < grp; ++k)
                if (NR > 0 || q0 + k < n) {
#pragma unroll
                    for (int h = 0; h < kSplit; ++h) widen(raw[k][h], x[h][k]);
                }
        }
#pragma unroll
        for (int k = 0; k < grp; ++k)
            if (NR > 0 || q0 + k < n) {
#pragma unroll
                for (int h = 0; h < kSplit; ++h)
#pragma unroll
                    for (int e = 0; e < kQuad; ++e)
                        g[h][e] = q0 + k == 0 ? x[h][k][e] : g[h][e] + x[h][k][e];
            }
    }
#pragma unroll
    for (int h = 0; h < kSplit; ++h) mean_clip(u, g[h]);
    return true;
}

// Writes a lane's quads of the output.
template <bool PB, Part PT, int POL>
__device__ __forceinline__ void store_part(Tensor &tn, int64_t i0, int lane,
                                           const float (&p)[kSplit][kQuad]) {
#pragma unroll
    for (int h = 0; h < kSplit; ++h) {
        const int off = kQuad * (lane + h * kWave);
        if constexpr (PT == kLast)
            store_quad<PB>(tn.out, i0 + off, tn.numel - (i0 + off), p[h]);
        else
            store_raw<PB, PT == kWhole, POL>(static_cast<char *>(tn.out) + i0 * (PB ? 2 : 4), off,
                                             narrow<PB>(p[h]));
    }
}

// Elements before the first at which every replica's quads are aligned, -1
// where the replicas do not share a phase.
template <bool GB>
__device__ __forceinline__ int common_head(Tensor &tn, int n) {
    constexpr uintptr_t es = GB ? 2 : 4;
    const int phase = (int)((uintptr_t)tn.grads[0] / es % kQuad);
    for (int q = 1; q < n; ++q)
        if ((int)((uintptr_t)tn.grads[q] / es % kQuad) != phase) return -1;
    return (kQuad - phase) % kQuad;
}

// Whether every stream of a part is aligned for whole-quad instructions. The
// group's values are asked for here as well, so that everything the table
// holds comes in one round trip: left to the branches that use it, it would
// come in a further one before the first gradient is asked for.
template <int NR, bool GB, bool PB>
__device__ __forceinline__ bool aligned_part(Tensor &tn, Group &gr, int nrep) {
    const int n = NR > 0 ? NR : nrep;
    uint32_t bits = (uint32_t)(uintptr_t)tn.out & (PB ? 7u : 15u);
    for (int q = 0; q < n; ++q) bits |= (uint32_t)(uintptr_t)tn.grads[q] & (GB ? 7u : 15u);
    asm volatile(""
                 : "+s"(bits)
                 : "s"(gr.decay), "s"(gr.factor), "s"(tn.numel), "s"(tn.piece0));
    return bits == 0;
}

// ------------------------------------------------------------ 32-bit states
// The moments (m, v updated in place) and the step they give.
__device__ __forceinline__ float moments32(float g, float &m, float &v, const Uniform &u) {
    m = __builtin_fmaf(g, u.sc.c1, m * u.sc.b1);
    v = __builtin_fmaf(u.sc.c2 * g, g, v * u.sc.b2);
    return (u.lr * (m / u.sc.bc1)) / (__builtin_sqrtf(v / u.sc.bc2) + u.sc.eps);
}

template <int NR, bool GB, bool PB, Part PT>
__device__ __forceinline__ void part32(const KernelArgs &a, Tensor &tn, Group &gr, int64_t i0,
                                       int64_t s0, int lane) {
    Uniform u;
    const span_t sp = span_of(a.st.master + s0, kWaveElems * 4);
    const span_t sm = span_of(a.st.m + s0, kWaveElems * 4);
    const span_t sv = span_of(a.st.v + s0, kWaveElems * 4);
    float g[kSplit][kQuad], p[kSplit][kQuad], m[kSplit][kQuad], v[kSplit][kQuad];
    const bool go = mean_part<NR, GB, PT>(tn, a.n, u, i0, lane, g, [&] {
#pragma unroll
        for (int h = 0; h < kSplit; ++h) {
            const int off = kQuad * (lane + h * kWave);
            load_f4<kPolNT>(sm, off, m[h]);
            load_f4<kPolNT>(sv, off, v[h]);
            if (!kLateMaster<NR, GB>) load_f4<kPolNT>(sp, off, p[h]);
        }
        __builtin_amdgcn_sched_barrier(0);
        return uniforms<NR>(a, gr, u);
    });
    if (!go) return;
    float d[kSplit][kQuad];
#pragma unroll
    for (int h = 0; h < kSplit; ++h)
#pragma unroll
        for (int e = 0; e < kQuad; ++e) d[h][e] = moments32(g[h][e], m[h][e], v[h][e], u);
    if (kLateMaster<NR, GB>) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int h = 0; h < kSplit; ++h) load_f4<kPolNT>(sp, kQuad * (lane + h * kWave), p[h]);
    }
#pragma unroll
    for (int h = 0; h < kSplit; ++h)
#pragma unroll
        for (int e = 0; e < kQuad; ++e) p[h][e] = p[h][e] * u.keep - d[h][e];
    if (PT == kLast) clear_behind(tn, i0, lane, p);
    const auto store = [&](auto pol) {
        constexpr int P = decltype(pol)::value;
#pragma unroll
        for (int h = 0; h < kSplit; ++h) store_f4<P>(sp, kQuad * (lane + h * kWave), p[h]);
#pragma unroll
        for (int h = 0; h < kSplit; ++h) store_f4<P>(sm, kQuad * (lane + h * kWave), m[h]);
#pragma unroll
        for (int h = 0; h < kSplit; ++h) store_f4<P>(sv, kQuad * (lane + h * kWave), v[h]);
        store_part<PB, PT, P>(tn, i0, lane, p);
    };
    if (a.stream_state) store(Const<kPolDevice>());
    else store(Const<kPolNT>());
}

template <int NR, bool GB, bool PB>
__global__ void __launch_bounds__(kWave) adamw32_kernel(KernelArgs a) {
    const int64_t piece = blockIdx.x / kPieceWaves;
    const int k = constant(a.map)[piece];
    Tensor &tn = constant(a.table)[k];
    Group &gr = constant(a.groups)[k];
    const bool al = aligned_part<NR, GB, PB>(tn, gr, a.n);
    const int64_t i0 = (piece - tn.piece0) * kAdamwPiece + (blockIdx.x % kPieceWaves) * kWaveElems;
    const int64_t s0 = (int64_t)blockIdx.x * kWaveElems;
    const int lane = threadIdx.x;
    if (i0 >= tn.numel) return;
    if (i0 + kWaveElems > tn.numel) part32<NR, GB, PB, kLast>(a, tn, gr, i0, s0, lane);
    else if (al) part32<NR, GB, PB, kWhole>(a, tn, gr, i0, s0, lane);
    else part32<NR, GB, PB, kUnaligned>(a, tn, gr, i0, s0, lane);
}

// ------------------------------------------------------------- 8-bit states
// e4m3 codes, 32 elements to a scale 2^(e - 127) held as the byte e. The
// largest finite magnitude of a block lies in (224, 448] scales (448 is the
// largest e4m3 value), or the scale is the smallest, 2^-126.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    const int e = (int)((top + 0x1FFFFFu) >> 23) - 8;   // + 1 above 1.75 * 2^E
    return e < 1 ? 1u : (uint32_t)e;
}
__device__ __forceinline__ float scale_of(uint32_t e) { return __uint_as_float(e << 23); }
__device__ __forceinline__ float scale_inv(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// Largest over the 8 lanes that hold a block, of magnitude bits (which order
// as the magnitudes do; an integer maximum takes its operand across lanes in
// the same instruction).
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
    const auto lane = [](uint32_t v, auto ctrl) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xF, 0xF,
                                                     false);
    };
    const auto larger = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    x = larger(x, lane(x, Const<0xB1>()));            // 1 lane apart
    x = larger(x, lane(x, Const<0x4E>()));            // 2 apart
    return larger(x, lane(x, Const<0x141>()));        // the other four
}

__device__ __forceinline__ bool finite(float x) {
    return (__float_as_uint(x) & 0x7FFFFFFFu) < 0x7F800000u;
}

// Largest magnitude of a quad. SAFE: what is not finite does not count, so
// an infinity or NaN of one element leaves its neighbours' codes alone.
template <bool SAFE>
__device__ __forceinline__ uint32_t quad_max(const float (&x)[kQuad]) {
    float t = 0.0f;
#pragma unroll
    for (int e = 0; e < kQuad; ++e)
        t = __builtin_fmaxf(t, SAFE && !finite(x[e]) ? 0.0f : __builtin_fabsf(x[e]));
    return __float_as_uint(t);
}

__device__ __forceinline__ uint32_t pack4(const float (&y)[kQuad]) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
}

__device__ __forceinline__ void unpack4(uint32_t w, float scale, float (&x)[kQuad]) {
    const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    x[0] = a.x * scale; x[1] = a.y * scale; x[2] = b.x * scale; x[3] = b.y * scale;
}

// r > 0 stays at least the smallest code, so a second moment that is there
// never becomes none: the median of y, that code and r times a large number,
// which is 0 for r = 0 and above every code otherwise (r, a root of a
// binary32 or what root() makes of one, is at least 2^-87).
__device__ __forceinline__ float at_least_a_code(float y, float r) {
    return __builtin_amdgcn_fmed3f(y, 0x1p-9f, r * 0x1p120f);
}

// A quad to codes on the scale 1/inv. `noise` (16 bits per element, its bit 15
// worth half a step) carries into the third mantissa bit and what is below is
// cut, which rounds without bias wherever e4m3 has three mantissa bits (2^-6
// scales and up); below, to nearest. SAFE: what is not finite becomes NaN;
// without it every value is finite.
template <bool ROOT, bool SAFE>
__device__ __forceinline__ uint32_t encode4(const float (&x)[kQuad], const uint32_t (&noise)[kQuad],
                                            float inv) {
    float y[kQuad];
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        y[e] = __uint_as_float((__float_as_uint(x[e]) + (noise[e] << 4)) & 0xFFF00000u) * inv;
        if (ROOT) y[e] = at_least_a_code(y[e], x[e]);
        if (SAFE && !finite(x[e])) y[e] = __builtin_nanf("");
    }
    return pack4(y);
}

struct Uniform8 : Uniform {
    float lrc, rs;
    uint32_t key;
};

template <int NR>
__device__ __forceinline__ bool uniforms8(const KernelArgs &a, Group &gr, Uniform8 &u) {
    if (!uniforms<NR>(a, gr, u)) return false;
    u.key = adamw_mix(a.seed ^ (a.sc_dev ? (uint32_t)(constant(a.ds)->t - 1) : a.t));
    u.lrc = u.lr * __builtin_amdgcn_rcpf(u.sc.bc1);      // 1 ulp, and so is the root
    u.rs = __builtin_amdgcn_rsqf(u.sc.bc2);
    return true;
}

// sqrt(v) from the hardware's reciprocal root (1 ulp) and one Newton step whose
// residue is exact: correctly rounded but for about one v in 2^21, off by one
// ulp there. A v below 2^-126 (gradients under 1e-18) gives less than its
// root, an infinite one NaN.
__device__ __forceinline__ float root(float v) {
    const float y = __builtin_amdgcn_rsqf(__builtin_fmaxf(v, 0x1p-126f));
    const float s = v * y;
    return __builtin_fmaf(__builtin_fmaf(-s, s, v), 0.5f * y, s);
}

// Fresh moments of a quad from the stored ones (codes cm, cr on the scales em,
// er), and the step d they give. b1 goes into m's scale, a power of two: the
// same bits as (code * scale) * b1 above the smallest scale. Only d takes the
// hardware's reciprocal (1 ulp; its operand is 0 or at least 2^-87): the
// codes do not depend on it.
__device__ __forceinline__ void moments8(const float (&g)[kQuad], uint32_t cm, uint32_t cr,
                                         uint32_t em, uint32_t er, float (&m)[kQuad],
                                         float (&r)[kQuad], float (&d)[kQuad], const Uniform8 &u) {
    unpack4(cm, scale_of(em) * u.sc.b1, m);
    unpack4(cr, scale_of(er), r);
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        m[e] = __builtin_fmaf(g[e], u.sc.c1, m[e]);
        r[e] = root(__builtin_fmaf(u.sc.c2 * g[e], g[e], (r[e] * r[e]) * u.sc.b2));
        d[e] = m[e] * __builtin_amdgcn_rcpf(__builtin_fmaf(r[e], u.rs, u.sc.eps));
    }
}

// Codes and scales of the quad q (its place in the state / 4).
template <bool SAFE>
__device__ __forceinline__ void encode8(const float (&m)[kQuad], const float (&r)[kQuad],
                                        const Uniform8 &u, int64_t q, uint32_t &cm, uint32_t &cr,
                                        uint32_t &em, uint32_t &er) {
    em = scale_byte(block_max(quad_max<SAFE>(m)));
    er = scale_byte(block_max(quad_max<SAFE>(r)));
    const uint32_t x = adamw_mix((uint32_t)q + (uint32_t)(q >> 32) * 0x7F4A7C15u + u.key);
    uint32_t w[kQuad] = {x, x * 0xB5297A4Du, x * 0x68E31DA5u, x * 0x1B56C4E9u};
    uint32_t nm[kQuad], nr[kQuad];
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        // opaque, or the compiler takes the low half's shift into a second
        // product (a product costs four of the other instructions)
        asm("" : "+v"(w[e]));
        nm[e] = w[e] >> 16;
        nr[e] = w[e] & 0xFFFFu;
    }
    cm = encode4<false, SAFE>(m, nm, scale_inv(em));
    cr = encode4<true, SAFE>(r, nr, scale_inv(er));
}

// Lanes with a step in their quad that is not finite, as it is where a moment
// is not (and where m/0 with eps = 0 is not, which costs time alone).
__device__ __forceinline__ uint64_t bad_lanes(const float (&d)[kQuad]) {
    uint64_t bad = 0;
#pragma unroll
    for (int e = 0; e < kQuad; ++e)
        bad |= __builtin_amdgcn_ballot_w64(!(__builtin_fabsf(d[e]) < __builtin_inff()));
    return bad;
}

template <int NR, bool GB, bool PB, Part PT>
__device__ __forceinline__ void part8(const KernelArgs &a, Tensor &tn, Group &gr, int64_t i0,
                                      int64_t s0, uint8_t *scale, int lane) {
    Uniform8 u;
    const span_t sp = span_of(a.st.master + s0, kWaveElems * 4);
    const span_t sm = span_of(a.st.m8 + s0, kWaveElems), sr = span_of(a.st.r8 + s0, kWaveElems);
    float g[kSplit][kQuad], p[kSplit][kQuad], m[kSplit][kQuad], r[kSplit][kQuad];
    uint32_t cm[kSplit], cr[kSplit], em[kSplit], er[kSplit];
    const bool go = mean_part<NR, GB, PT>(tn, a.n, u, i0, lane, g, [&] {
#pragma unroll
        for (int h = 0; h < kSplit; ++h) {
            const int off = kQuad * (lane + h * kWave);
            cm[h] = __builtin_amdgcn_raw_buffer_load_b32(sm, off, 0, kPolNT);
            cr[h] = __builtin_amdgcn_raw_buffer_load_b32(sr, off, 0, kPolNT);
            em[h] = scale[off / kAdamwBlock];
            er[h] = scale[kAdamwScales + off / kAdamwBlock];
            if (!kLateMaster<NR, GB>) load_f4<kPolNT>(sp, off, p[h]);
        }
        __builtin_amdgcn_sched_barrier(0);
        return uniforms8<NR>(a, gr, u);
    });
    if (!go) return;
    float d[kSplit][kQuad];
    uint64_t bad = 0;
#pragma unroll
    for (int h = 0; h < kSplit; ++h) {
        moments8(g[h], cm[h], cr[h], em[h], er[h], m[h], r[h], d[h], u);
        bad |= bad_lanes(d[h]);
    }
    const int64_t q = s0 / kQuad + lane;
    if (__builtin_expect(bad != 0, 0)) {
#pragma unroll
        for (int h = 0; h < kSplit; ++h)
            encode8<true>(m[h], r[h], u, q + h * kWave, cm[h], cr[h], em[h], er[h]);
    } else {
#pragma unroll
        for (int h = 0; h < kSplit; ++h)
            encode8<false>(m[h], r[h], u, q + h * kWave, cm[h], cr[h], em[h], er[h]);
    }
    if (kLateMaster<NR, GB>) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int h = 0; h < kSplit; ++h) load_f4<kPolNT>(sp, kQuad * (lane + h * kWave), p[h]);
    }
#pragma unroll
    for (int h = 0; h < kSplit; ++h)
#pragma unroll
        for (int e = 0; e < kQuad; ++e)
            p[h][e] = __builtin_fmaf(-u.lrc, d[h][e], p[h][e] * u.keep);
    if (PT == kLast) clear_behind(tn, i0, lane, p);
    const auto store = [&](auto pol) {
        constexpr int P = decltype(pol)::value;
#pragma unroll
        for (int h = 0; h < kSplit; ++h) {
            const int off = kQuad * (lane + h * kWave);
            store_f4<P>(sp, off, p[h]);
            __builtin_amdgcn_raw_buffer_store_b32(cm[h], sm, off, 0, P);
            __builtin_amdgcn_raw_buffer_store_b32(cr[h], sr, off, 0, P);
        }
        store_part<PB, PT, P>(tn, i0, lane, p);
    };
    if (a.stream_state) store(Const<kPolDevice>());
    else store(Const<kPolNT>());
    if (lane % (kAdamwBlock / kQuad) == 0) {
#pragma unroll
        for (int h = 0; h < kSplit; ++h) {
            const int blk = kQuad * (lane + h * kWave) / kAdamwBlock;
            scale[blk] = (uint8_t)em[h];
            scale[kAdamwScales + blk] = (uint8_t)er[h];
        }
    }
}

template <int NR, bool GB, bool PB>
__global__ void __launch_bounds__(kWave *kPieceWaves) adamw8_kernel(KernelArgs a) {
    const int64_t piece = blockIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lane = threadIdx.x % kWave;
    const int k = constant(a.map)[piece];
    Tensor &tn = constant(a.table)[k];
    Group &gr = constant(a.groups)[k];
    const bool al = aligned_part<NR, GB, PB>(tn, gr, a.n);
    const int64_t i0 = (piece - tn.piece0) * kAdamwPiece + wave * kWaveElems;
    const int64_t s0 = piece * kAdamwPiece + wave * kWaveElems;
    uint8_t *scale = a.st.scale + piece * (2 * kAdamwScales) + wave * (kWaveElems / kAdamwBlock);
    if (i0 >= tn.numel) return;
    if (i0 + kWaveElems > tn.numel) part8<NR, GB, PB, kLast>(a, tn, gr, i0, s0, scale, lane);
    else if (al) part8<NR, GB, PB, kWhole>(a, tn, gr, i0, s0, scale, lane);
    else part8<NR, GB, PB, kUnaligned>(a, tn, gr, i0, s0, scale, lane);
}

// m and v = r*r of a piece in fp32 (r has four significant bits, so its
// square is exact), and back: codes to nearest, ties to even, on the same
// scales. Values that came from codes map to codes of the same values.
__global__ void __launch_bounds__(256)
adamw_decode_kernel(AdamwStateRef st, float *m, float *v) {
    const int64_t piece = blockIdx.x;
    const uint8_t *scale = st.scale + piece * (2 * kAdamwScales);
    for (int k = threadIdx.x; k < kAdamwPiece / kQuad; k += 256) {
        const int64_t i = piece * kAdamwPiece + kQuad * k;
        const int blk = kQuad * k / kAdamwBlock;
        float x[kQuad];
        if (m) {
            unpack4(*reinterpret_cast<const uint32_t *>(st.m8 + i), scale_of(scale[blk]), x);
            __builtin_memcpy(m + i, x, sizeof x);        // the caller's alignment
        }
        if (v) {
            unpack4(*reinterpret_cast<const uint32_t *>(st.r8 + i),
                    scale_of(scale[kAdamwScales + blk]), x);
#pragma unroll
            for (int e = 0; e < kQuad; ++e) x[e] = x[e] * x[e];
            __builtin_memcpy(v + i, x, sizeof x);
        }
    }
}

template <bool ROOT>
__device__ __forceinline__ void encode_nearest(const float *src, uint8_t *codes, uint8_t *scale,
                                               int k) {
    float x[kQuad];
    __builtin_memcpy(x, src + kQuad * k, sizeof x);
#pragma unroll
    for (int e = 0; e < kQuad; ++e)
        if (ROOT) x[e] = __builtin_sqrtf(x[e]);
    const uint32_t eb = scale_byte(block_max(quad_max<true>(x)));
    const float inv = scale_inv(eb);
    float y[kQuad];
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        y[e] = x[e] * inv;
        if (ROOT) y[e] = at_least_a_code(y[e], x[e]);
        if (!finite(x[e])) y[e] = __builtin_nanf("");
    }
    *reinterpret_cast<uint32_t *>(codes + kQuad * k) = pack4(y);
    if (k % (kAdamwBlock / kQuad) == 0) scale[kQuad * k / kAdamwBlock] = (uint8_t)eb;
}

__global__ void __launch_bounds__(256)
adamw_encode_kernel(AdamwStateRef st, const float *m, const float *v) {
    const int64_t piece = blockIdx.x, i = piece * kAdamwPiece;
    uint8_t *scale = st.scale + piece * (2 * kAdamwScales);
    for (int k = threadIdx.x; k < kAdamwPiece / kQuad; k += 256) {   // whole waves
        if (m) encode_nearest<false>(m + i, st.m8 + i, scale, k);
        if (v) encode_nearest<true>(v + i, st.r8 + i, scale + kAdamwScales, k);
    }
}

__global__ void __launch_bounds__(256) adamw_clear_kernel(AdamwStateRef st) {
    const int64_t piece = blockIdx.x;
    for (int k = threadIdx.x; k < kAdamwPiece / kQuad; k += 256) {
        reinterpret_cast<uint32_t *>(st.m8 + piece * kAdamwPiece)[k] = 0u;
        reinterpret_cast<uint32_t *>(st.r8 + piece * kAdamwPiece)[k] = 0u;
    }
    if (threadIdx.x < 2 * kAdamwScales) st.scale[piece * (2 * kAdamwScales) + threadIdx.x] = 1;
}

template <bool FB>
__global__ void __launch_bounds__(256) widen_kernel(const void *src, float *dst, int64_t n) {
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += stride)
        dst[i] = elem<FB>(src, i);
}

// ----------------------------------------------------------- sum of squares
// S = sum over all elements of (sum_q g_q)^2 / N^2, everything in binary64.
// Wave w takes pieces w, w + W, ...; a workgroup's partial sum goes to memory and
// the last workgroup to finish adds the partials in their order, so the
// result does not depend on which one that is. Which wave and lane takes an
// element depends on the sizes and on the replicas' common phase (common_head).
constexpr int kSumsqBlock = 256;
constexpr int kRow = kQuad * kWave;              // elements that a wave reads in one turn

__device__ __forceinline__ double wave_sum(double x) {
    for (int d = kWave / 2; d > 0; d /= 2) x += __shfl_xor(x, d);
    return x;
}

__device__ __forceinline__ double group_sum(double x, double *lds) {
    x = wave_sum(x);
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = x;
    __syncthreads();
    double s = 0.0;
    for (int k = 0; k < kSumsqBlock / kWave; ++k) s += lds[k];
    __syncthreads();
    return s;
}

// Squares of TURNS rows of 256 elements from element i0 on, a quad per lane
// and row, all rows in flight together.
template <int NR, bool GB, int TURNS, bool AL>
__device__ __forceinline__ double squares_rows(Tensor &tn, int nrep, int64_t i0,
                                               int lane) {
    const int n = NR > 0 ? NR : nrep;
    constexpr int es = GB ? 2 : 4;
    constexpr int grp = kGroupOf<NR>;
    double s[TURNS][kQuad];
#pragma unroll 1
    for (int q0 = 0; q0 < n; q0 += grp) {
        RawQuad<GB> raw[grp][TURNS];
#pragma unroll
        for (int k = 0; k < grp; ++k)
            if (NR > 0 || q0 + k < n) {
                const char *base = static_cast<const char *>(tn.grads[q0 + k]) + i0 * es;
#pragma unroll
                for (int h = 0; h < TURNS; ++h)
                    raw[k][h] = load_raw<GB, AL, kPolNT>(base, kQuad * (lane + h * kWave));
            }
#pragma unroll
        for (int k = 0; k < grp; ++k)
            if (NR > 0 || q0 + k < n) {
#pragma unroll
                for (int h = 0; h < TURNS; ++h) {
                    float x[kQuad];
                    widen(raw[k][h], x);
#pragma unroll
                    for (int e = 0; e < kQuad; ++e)
                        s[h][e] = q0 + k == 0 ? (double)x[e] : s[h][e] + (double)x[e];
                }
            }
    }
    double acc = 0.0;
#pragma unroll
    for (int h = 0; h < TURNS; ++h)
#pragma unroll
        for (int e = 0; e < kQuad; ++e) acc = __builtin_fma(s[h][e], s[h][e], acc);
    return acc;
}

// Squares of what a tensor has from element i0 on, less than a piece: whole
// rows 4, 2 and 1 at a time, then the last one. Taking a row and a replica at
// a time instead waits for memory once for each: 48 layers of width 129, half
// of the rows, bf16: 11.3 us against 14.6 with four replicas, 6.4 against 7.2
// with one.
template <int NR, bool GB>
__device__ __forceinline__ double squares_last(Tensor &tn, int nrep, int64_t i0, int lane) {
    const int n = NR > 0 ? NR : nrep;
    constexpr int grp = kGroupOf<NR>;
    double acc = 0.0;
    for (; i0 + 4 * kRow <= tn.numel; i0 += 4 * kRow)
        acc += squares_rows<NR, GB, 4, false>(tn, n, i0, lane);
    if (i0 + 2 * kRow <= tn.numel) {
        acc += squares_rows<NR, GB, 2, false>(tn, n, i0, lane);
        i0 += 2 * kRow;
    }
    if (i0 + kRow <= tn.numel) {
        acc += squares_rows<NR, GB, 1, false>(tn, n, i0, lane);
        i0 += kRow;
    }
    const int64_t i = i0 + kQuad * lane;
    if (i >= tn.numel) return acc;
    double s[kQuad];
#pragma unroll 1
    for (int q0 = 0; q0 < n; q0 += grp) {
        float x[grp][kQuad];
        load_last<NR, GB>(tn, q0, n, i, tn.numel - i, x);
#pragma unroll
        for (int k = 0; k < grp; ++k)
            if (NR > 0 || q0 + k < n) {
#pragma unroll
                for (int e = 0; e < kQuad; ++e)
                    s[e] = q0 + k == 0 ? (double)x[k][e] : s[e] + (double)x[k][e];
            }
    }
#pragma unroll
    for (int e = 0; e < kQuad; ++e) acc = __builtin_fma(s[e], s[e], acc);
    return acc;
}

// Whether workgroup b is the last of n to come here. Counting on one address
// serialises (about 10 ns each: 10.4 us for 3M elements against 6.3 us), so
// workgroups count on the counter of b mod kSumsqCounters, and the last one of
// each on the one behind them. A full counter goes back to 0.
__device__ __forceinline__ bool last_of(uint32_t *done, unsigned b, unsigned n) {
    const auto full = [](uint32_t *c, unsigned want) {
        if (__hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != want - 1)
            return false;
        __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return true;
    };
    constexpr unsigned split = kSumsqCounters;
    const unsigned c = b % split;
    return full(done + c * kSumsqCounterWords, n / split + (c < n % split ? 1 : 0)) &&
           full(done + split * kSumsqCounterWords, n < split ? n : split);
}

template <int NR, bool GB>
__global__ void __launch_bounds__(kSumsqBlock)
sumsq_kernel(const AdamwTensor *table, const int32_t *map,
             int64_t npieces, int nrep, double *partial, uint32_t *done, double *out) {
    __shared__ double lds[kSumsqBlock / kWave];
    __shared__ bool last;
    const int n = NR > 0 ? NR : nrep;
    // quads of a lane in flight together: 64 of bf16 or 32 of fp32 over the
    // replicas, at most 8 of each (two workgroups per unit leave each wave
    // 256 registers)
    constexpr int width = NR == 0 || NR > kGroup ? kGroup : NR;
    constexpr int flight = GB ? 64 : 32;
    // three of fp32 by 4, not 8: odd widths 55.5 us against 63.0, GPT-2 small's
    // rank 31.5 against 36.3, Llama-7B list 1.46 ms against 1.50
    constexpr int turns = !GB && NR == 3 ? 4 : flight / width >= 8 ? 8 : flight / width;
    static_assert(kAdamwPiece % (turns * kRow) == 0, "whole rounds in a piece");
    const int lane = threadIdx.x % kWave;
    const int64_t first = (int64_t)blockIdx.x * (kSumsqBlock / kWave) +
                          __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    double acc = 0.0;
    const int64_t stride = (int64_t)gridDim.x * (kSumsqBlock / kWave);
    int k = first < npieces ? constant(map)[first] : 0;
    for (int64_t piece = first; piece < npieces; piece += stride) {
        Tensor &tn = constant(table)[k];
        // the next piece's tensor, in the round trip of this one's entry
        k = piece + stride < npieces ? constant(map)[piece + stride] : k;
        asm volatile("" : "+s"(k) : "s"(tn.numel), "s"(tn.piece0), "s"(tn.grads[0]));
        // The windows that waves read start `head` elements into the tensor's
        // pieces, where all replicas are aligned if they share a phase (44 us
        // against 36 without, three bf16 replicas of 28M elements, 3 elements
        // off); the first wave takes the head.
        const int head = common_head<GB>(tn, n);
        const bool al = head >= 0;
        int64_t i0 = (piece - tn.piece0) * kAdamwPiece;
        if (al) {
            if (i0 == 0 && lane < head && lane < tn.numel) {
                double s = 0.0;
                for (int q = 0; q < n; ++q) s += (double)elem<GB>(tn.grads[q], lane);
                acc = __builtin_fma(s, s, acc);
            }
            i0 += head;
        }
        if (i0 + kAdamwPiece <= tn.numel) {
            for (int h = 0; h < kAdamwPiece; h += turns * kRow)
                acc += al ? squares_rows<NR, GB, turns, true>(tn, n, i0 + h, lane)
                          : squares_rows<NR, GB, turns, false>(tn, n, i0 + h, lane);
        } else {
            acc += squares_last<NR, GB>(tn, n, i0, lane);
        }
    }
    const double s = group_sum(acc, lds);
    if (threadIdx.x == 0) {
        __hip_atomic_store(&partial[blockIdx.x], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        // The partial is the only thing to be ordered before the count.
        // This holds on gfx950 and leans on its instructions, not on the
        // language's memory model: an agent-scope store (sc1) writes through
        // and is acknowledged once every XCD can see it, so waiting for it is
        // enough, and the joining workgroup's agent-scope loads (sc1) read
        // past its own caches. A release and acquire at the counter would
        // write back and drop the whole L2 in every workgroup: 139 us against
        // 52 us (15.6M elements, N = 8, bf16, 2048 workgroups).
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        last = last_of(done, blockIdx.x, gridDim.x);
    }
    __syncthreads();
    if (!last) return;
    constexpr int per = kSumsqGroups / kSumsqBlock;       // all loads in flight together
    double x[per], t = 0.0;
#pragma unroll
    for (int k = 0; k < per; ++k) {
        const unsigned i = threadIdx.x + k * kSumsqBlock;
        x[k] = i < gridDim.x ? __hip_atomic_load(&partial[i], __ATOMIC_RELAXED,
                                                 __HIP_MEMORY_SCOPE_AGENT) : 0.0;
    }
#pragma unroll
    for (int k = 0; k < per; ++k) t += x[k];
    t = group_sum(t, lds);
    if (threadIdx.x == 0) {
        *out = t / ((double)n * (double)n);
    }
}

template <int NR, bool GB, bool PB>
hipError_t launch_typed(const AdamwArgs &a, hipStream_t stream) {
    KernelArgs k = {a.table, a.groups, a.map, a.n, a.st, a.sc, a.sc_dev, a.ds, a.seed, a.t, a.sumsq,
                    a.max_norm, a.stream_state ? 1 : 0};
    if (a.q8)
        hipLaunchKernelGGL((adamw8_kernel<NR, GB, PB>), dim3((unsigned)a.npieces),
                           dim3(kWave * kPieceWaves), kLds8, stream, k);
    else
        hipLaunchKernelGGL((adamw32_kernel<NR, GB, PB>), dim3((unsigned)(a.npieces * kPieceWaves)),
                           dim3(kWave), kLds32, stream, k);
    return hipGetLastError();
}

template <bool GB, bool PB>
hipError_t launch_replicas(const AdamwArgs &a, hipStream_t stream) {
    switch (a.n) {
    case 1: return launch_typed<1, GB, PB>(a, stream);
    case 2: return launch_typed<2, GB, PB>(a, stream);
    case 4: return launch_typed<4, GB, PB>(a, stream);
    case 8: return launch_typed<8, GB, PB>(a, stream);
    default: return launch_typed<0, GB, PB>(a, stream);
    }
}

template <int NR, bool GB>
hipError_t sumsq_typed(const SumsqArgs &a, hipStream_t stream) {
    constexpr int per = kSumsqBlock / kWave;
    const int64_t groups = (a.npieces + per - 1) / per;
    int64_t grid = groups < kSumsqGroups ? groups : kSumsqGroups;
    if (grid < 1) grid = 1;                     // no elements: a sum of zero
    hipLaunchKernelGGL((sumsq_kernel<NR, GB>), dim3((unsigned)grid), dim3(kSumsqBlock), 0, stream,
                       a.table, a.map, a.npieces, a.n, a.partial, a.done, a.out);
    return hipGetLastError();
}

// Replica counts known when compiled, against the count of the run (us; odd
// widths, GPT-2 small's rank 3 of 8, Llama-7B list's rank 0 of 8):
//            bf16                                        fp32
//   1   13.1 15.6    8.7 10.4    229 279       20.2 21.7   12.6 14.2    482 471
//   2   22.3 23.6   13.6 14.7    470 476       39.6 38.5   23.5 22.2    940 973
//   3   31.6 32.8   18.5 19.0    723 715       55.5 56.0   31.5 31.7   1456 1459
//   4   40.2 41.7   23.9 24.2    982 975       71.2 74.0   40.5 42.8   1925 1955
//   8   76.2 77.9   42.4 45.8   1898 1918     144.0 143.9  81.1 81.0   3892 3883
// Eleven tensors of 893 elements in all, four of fp32: 4.4 and 5.7.
template <bool GB>
hipError_t sumsq_replicas(const SumsqArgs &a, hipStream_t stream) {
    switch (a.n) {
    case 1: return sumsq_typed<1, GB>(a, stream);
    case 2: return sumsq_typed<2, GB>(a, stream);
    case 3: return sumsq_typed<3, GB>(a, stream);
    case 4: return sumsq_typed<4, GB>(a, stream);
    case 8: return sumsq_typed<8, GB>(a, stream);
    default: return sumsq_typed<0, GB>(a, stream);
    }
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs &a, hipStream_t stream) {
    if (a.n < 1 || a.n > kAdamwMaxReplicas) return hipErrorInvalidValue;
    if (a.npieces <= 0) return hipSuccess;
    if (a.npieces > kAdamwMaxPieces) return hipErrorInvalidConfiguration;
    if (a.grad_bf16)
        return a.out_bf16 ? launch_replicas<true, true>(a, stream)
                          : launch_replicas<true, false>(a, stream);
    return a.out_bf16 ? launch_replicas<false, true>(a, stream)
                      : launch_replicas<false, false>(a, stream);
}

hipError_t launch_sumsq(const SumsqArgs &a, hipStream_t stream) {
    if (a.n < 1 || a.n > kAdamwMaxReplicas) return hipErrorInvalidValue;
    return a.grad_bf16 ? sumsq_replicas<true>(a, stream) : sumsq_replicas<false>(a, stream);
}

hipError_t launch_adamw_decode(const AdamwStateRef &st, int64_t npieces, float *m, float *v,
                               hipStream_t stream) {
    if (npieces <= 0 || (!m && !v)) return hipSuccess;
    hipLaunchKernelGGL(adamw_decode_kernel, dim3((unsigned)npieces), dim3(256), 0, stream, st, m, v);
    return hipGetLastError();
}

hipError_t launch_adamw_encode(const AdamwStateRef &st, int64_t npieces, const float *m,
                               const float *v, hipStream_t stream) {
    if (npieces <= 0 || (!m && !v)) return hipSuccess;
    hipLaunchKernelGGL(adamw_encode_kernel, dim3((unsigned)npieces), dim3(256), 0, stream, st, m, v);
    return hipGetLastError();
}

hipError_t launch_adamw_clear(const AdamwStateRef &st, int64_t npieces, hipStream_t stream) {
    if (npieces <= 0) return hipSuccess;
    hipLaunchKernelGGL(adamw_clear_kernel, dim3((unsigned)npieces), dim3(256), 0, stream, st);
    return hipGetLastError();
}

hipError_t launch_widen(const void *src, bool src_bf16, float *master, int64_t n,
                        hipStream_t stream) {
    if (n <= 0) return hipSuccess;
    const int64_t want = (n + 255) / 256;
    const dim3 g((unsigned)(want < 65536 ? want : 65536)), b(256);
    if (src_bf16) hipLaunchKernelGGL(widen_kernel<true>, g, b, 0, stream, src, master, n);
    else hipLaunchKernelGGL(widen_kernel<false>, g, b, 0, stream, src, master, n);
    return hipGetLastError();
}

}  // namespace zk
