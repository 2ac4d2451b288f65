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
//     p = p * keep_k - ((lr_k / bc1) * m) / (r * (1/sqrt(bc2)) + eps)
// with bc = 1 - b^t. The 32-bit step without decay and clipping is bit for
// bit the per-parameter step of zero_kernels.hip.
//
// All of it is bound by HBM (about one operation per byte at one replica).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_internal.h"

namespace zk {

namespace {

constexpr int kWave = 64;
constexpr int kQuad = 4;                         // elements per lane and load
constexpr int kWaveElems = 8 * kWave;            // a wave's part of a piece
constexpr int kPieceWaves = kAdamwPiece / kWaveElems;

__device__ __forceinline__ float widen_bf16(uint32_t bits16) {
    return __uint_as_float(bits16 << 16);
}

// binary32 -> bf16 bits, round to nearest, ties to even; NaN stays NaN.
__device__ __forceinline__ uint32_t round_bf16(float x) {
    uint32_t u = __float_as_uint(x);
    uint32_t r = (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
    return ((u & 0x7FFFFFFFu) > 0x7F800000u) ? ((u >> 16) | 0x40u) : r;
}

template <bool B>
__device__ __forceinline__ float elem(const void *base, int64_t i) {
    return B ? widen_bf16(static_cast<const uint16_t *>(base)[i])
             : static_cast<const float *>(base)[i];
}

// Elements [i, i + 4) of a gradient at its own alignment; `left` of them
// exist, the others are zero.
template <bool B>
__device__ __forceinline__ void load_quad(const void *base, int64_t i, int64_t left,
                                          float (&x)[kQuad]) {
    if (left >= kQuad) {
        if constexpr (B) {
            uint2 w;
            __builtin_memcpy(&w, static_cast<const uint16_t *>(base) + i, sizeof w);
            x[0] = widen_bf16(w.x & 0xFFFFu);
            x[1] = widen_bf16(w.x >> 16);
            x[2] = widen_bf16(w.y & 0xFFFFu);
            x[3] = widen_bf16(w.y >> 16);
        } else {
            float4 w;
            __builtin_memcpy(&w, static_cast<const float *>(base) + i, sizeof w);
            x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kQuad; ++e) x[e] = e < left ? elem<B>(base, i + e) : 0.0f;
    }
}

template <bool B>
__device__ __forceinline__ void store_quad(void *base, int64_t i, int64_t left,
                                           const float (&x)[kQuad]) {
    if (left >= kQuad) {
        if constexpr (B) {
            const uint2 w = make_uint2(round_bf16(x[0]) | (round_bf16(x[1]) << 16),
                                       round_bf16(x[2]) | (round_bf16(x[3]) << 16));
            __builtin_memcpy(static_cast<uint16_t *>(base) + i, &w, sizeof w);
        } else {
            const float4 w = make_float4(x[0], x[1], x[2], x[3]);
            __builtin_memcpy(static_cast<float *>(base) + i, &w, sizeof w);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kQuad; ++e) {
            if (e < left) {
                if (B) static_cast<uint16_t *>(base)[i + e] = (uint16_t)round_bf16(x[e]);
                else static_cast<float *>(base)[i + e] = x[e];
            }
        }
    }
}

struct KernelArgs {
    const AdamwTensor *__restrict__ table;
    const int32_t *__restrict__ map;
    int n;
    AdamwStateRef st;
    StepScalars sc;
    const StepScalars *sc_dev;
    const DevSchedule *ds;
    uint32_t seed, t;
    const double *sumsq;
    double max_norm;
};

// The clip factor; false where the sum of squares is not finite, and then
// the step writes nothing.
__device__ __forceinline__ bool clip_factor(const double *sumsq, double max_norm, float &c) {
    c = 1.0f;
    if (!sumsq) return true;
    const double s = *sumsq;
    if (!(s >= 0.0 && s < __builtin_inf())) return false;
    const double f = max_norm / (__builtin_sqrt(s) + 1e-6);
    if (f < 1.0) c = (float)f;
    return true;
}

// Mean gradient of a lane's quad, clipped.
template <int NR, bool GB>
__device__ __forceinline__ void mean_quad(const AdamwTensor &tn, const KernelArgs &a, float clip,
                                          int64_t i, int64_t left, float (&g)[kQuad]) {
    const int n = NR > 0 ? NR : a.n;
    const bool pow2 = NR > 0 ? (NR & (NR - 1)) == 0 : a.sc.n_pow2 != 0;
    load_quad<GB>(tn.grads[0], i, left, g);
#pragma unroll
    for (int q = 1; q < n; ++q) {
        float x[kQuad];
        load_quad<GB>(tn.grads[q], i, left, x);
#pragma unroll
        for (int e = 0; e < kQuad; ++e) g[e] = g[e] + x[e];
    }
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        // the replica count is the binding's, also where the schedule's
        // scalars come from the device
        g[e] = pow2 ? g[e] * a.sc.inv_n : g[e] / a.sc.nf;
        g[e] = g[e] * clip;
    }
}

// ------------------------------------------------------------ 32-bit states
template <int NR, bool GB, bool PB>
__global__ void __launch_bounds__(kWave) adamw32_kernel(KernelArgs a) {
    const int64_t piece = blockIdx.x / kPieceWaves;
    const AdamwTensor &tn = a.table[a.map[piece]];
    const int64_t numel = tn.numel;
    const int64_t i0 = (piece - tn.piece0) * kAdamwPiece + (blockIdx.x % kPieceWaves) * kWaveElems;
    if (i0 >= numel) return;
    float clip;
    if (!clip_factor(a.sumsq, a.max_norm, clip)) return;
    const StepScalars sc = a.sc_dev ? *a.sc_dev : a.sc;
    const float lr = sc.lr * tn.factor;
    const float keep = 1.0f - lr * tn.decay;
    const int64_t s0 = (int64_t)blockIdx.x * kWaveElems;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int off = kQuad * (threadIdx.x + h * kWave);
        const int64_t left = numel - (i0 + off);
        if (left <= 0) continue;
        float g[kQuad];
        mean_quad<NR, GB>(tn, a, clip, i0 + off, left, g);
        float4 *pp = reinterpret_cast<float4 *>(a.st.master + s0 + off);
        float4 *pm = reinterpret_cast<float4 *>(a.st.m + s0 + off);
        float4 *pv = reinterpret_cast<float4 *>(a.st.v + s0 + off);
        const float4 p4 = *pp, m4 = *pm, v4 = *pv;
        float p[kQuad] = {p4.x, p4.y, p4.z, p4.w};
        float m[kQuad] = {m4.x, m4.y, m4.z, m4.w};
        float v[kQuad] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int e = 0; e < kQuad; ++e) {
            const float mm = __builtin_fmaf(g[e], sc.c1, m[e] * sc.b1);
            const float vv = __builtin_fmaf(sc.c2 * g[e], g[e], v[e] * sc.b2);
            const float u = (lr * (mm / sc.bc1)) / (__builtin_sqrtf(vv / sc.bc2) + sc.eps);
            const bool in = e < left;
            p[e] = in ? p[e] * keep - u : 0.0f;
            m[e] = in ? mm : 0.0f;
            v[e] = in ? vv : 0.0f;
        }
        *pp = make_float4(p[0], p[1], p[2], p[3]);
        *pm = make_float4(m[0], m[1], m[2], m[3]);
        *pv = make_float4(v[0], v[1], v[2], v[3]);
        store_quad<PB>(tn.out, i0 + off, left, p);
    }
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

// Largest over the 8 lanes that hold a block.
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
    uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, false);
    x = x > y ? x : y;                                   // lanes 1 apart
    y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, false);
    x = x > y ? x : y;                                   // 2 apart
    y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, false);
    return x > y ? x : y;                                // the other four
}

constexpr uint32_t kInfBits = 0x7F800000u;

// Magnitude bits for the block's maximum: what is not finite does not count,
// so an infinity or NaN of one element leaves its neighbours' codes alone.
__device__ __forceinline__ uint32_t top_bits(float x) {
    const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
    return u < kInfBits ? u : 0u;
}

__device__ __forceinline__ uint32_t pack4(const float (&y)[kQuad]) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
}

typedef float f32x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void unpack4(uint32_t w, float scale, float (&x)[kQuad]) {
    const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    x[0] = a.x * scale; x[1] = a.y * scale; x[2] = b.x * scale; x[3] = b.y * scale;
}

// A quad to codes. `noise` (16 bits per element, its bit 15 worth half a
// step) carries into the third mantissa bit and what is below is cut, which
// rounds without bias wherever e4m3 has three mantissa bits (2^-6 scales and
// up); below, to nearest. ROOT: r > 0 stays at least the smallest code, so a
// moment that is there never becomes none. Not finite: NaN.
template <bool ROOT>
__device__ __forceinline__ uint32_t encode4(const float (&x)[kQuad], const uint32_t (&noise)[kQuad],
                                            float inv) {
    float y[kQuad];
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        const uint32_t u = __float_as_uint(x[e]);
        y[e] = __uint_as_float((u + (noise[e] << 4)) & 0xFFF00000u) * inv;
        if (ROOT) y[e] = x[e] > 0.0f ? __builtin_fmaxf(y[e], 0x1p-9f) : y[e];
        if ((u & 0x7FFFFFFFu) >= kInfBits) y[e] = __builtin_nanf("");
    }
    return pack4(y);
}

template <int NR, bool GB, bool PB>
__global__ void __launch_bounds__(kWave *kPieceWaves) adamw8_kernel(KernelArgs a) {
    const int64_t piece = blockIdx.x;
    const AdamwTensor &tn = a.table[a.map[piece]];
    const int64_t numel = tn.numel;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int64_t i0 = (piece - tn.piece0) * kAdamwPiece + wave * kWaveElems;
    if (i0 >= numel) return;
    float clip;
    if (!clip_factor(a.sumsq, a.max_norm, clip)) return;
    const StepScalars sc = a.sc_dev ? *a.sc_dev : a.sc;
    const uint32_t key = adamw_mix(a.seed ^ (a.sc_dev ? (uint32_t)(a.ds->t - 1) : a.t));
    const float lr = sc.lr * tn.factor;
    const float keep = 1.0f - lr * tn.decay;
    const float lrc = lr / sc.bc1;
    const float rs = 1.0f / __builtin_sqrtf(sc.bc2);
    const int64_t s0 = piece * kAdamwPiece + wave * kWaveElems;
    uint8_t *scale = a.st.scale + piece * (2 * kAdamwScales) + wave * (kWaveElems / kAdamwBlock);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int off = kQuad * (lane + h * kWave);
        const int blk = off / kAdamwBlock;
        // elements past the last read as zero and stay zero
        const int64_t left = numel - (i0 + off);
        float g[kQuad] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (left > 0) mean_quad<NR, GB>(tn, a, clip, i0 + off, left, g);
        uint32_t *cm = reinterpret_cast<uint32_t *>(a.st.m8 + s0 + off);
        uint32_t *cr = reinterpret_cast<uint32_t *>(a.st.r8 + s0 + off);
        float4 *pp = reinterpret_cast<float4 *>(a.st.master + s0 + off);
        const float4 p4 = *pp;
        float p[kQuad] = {p4.x, p4.y, p4.z, p4.w}, m[kQuad], r[kQuad];
        unpack4(*cm, scale_of(scale[blk]), m);
        unpack4(*cr, scale_of(scale[kAdamwScales + blk]), r);
        uint32_t tm = 0, tr = 0;
#pragma unroll
        for (int e = 0; e < kQuad; ++e) {
            m[e] = __builtin_fmaf(g[e], sc.c1, m[e] * sc.b1);
            const float v = __builtin_fmaf(sc.c2 * g[e], g[e], (r[e] * r[e]) * sc.b2);
            r[e] = __builtin_sqrtf(v);
            p[e] = p[e] * keep - (lrc * m[e]) / (r[e] * rs + sc.eps);
            if (e >= left) p[e] = 0.0f;                 // 0/0 where eps is 0
            const uint32_t bm = top_bits(m[e]), br = top_bits(r[e]);
            tm = tm > bm ? tm : bm;
            tr = tr > br ? tr : br;
        }
        const uint32_t em = scale_byte(block_max(tm)), er = scale_byte(block_max(tr));
        const int64_t q = (s0 + off) / kQuad;
        const uint32_t x = adamw_mix((uint32_t)q + (uint32_t)(q >> 32) * 0x7F4A7C15u + key);
        const uint32_t w[kQuad] = {x, x * 0xB5297A4Du, x * 0x68E31DA5u, x * 0x1B56C4E9u};
        uint32_t nm[kQuad], nr[kQuad];
#pragma unroll
        for (int e = 0; e < kQuad; ++e) {
            nm[e] = w[e] >> 16;
            nr[e] = w[e] & 0xFFFFu;
        }
        *cm = encode4<false>(m, nm, scale_inv(em));
        *cr = encode4<true>(r, nr, scale_inv(er));
        *pp = make_float4(p[0], p[1], p[2], p[3]);
        if (lane % (kAdamwBlock / kQuad) == 0) {
            scale[blk] = (uint8_t)em;
            scale[kAdamwScales + blk] = (uint8_t)er;
        }
        if (left > 0) store_quad<PB>(tn.out, i0 + off, left, p);
    }
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
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        if (ROOT) x[e] = __builtin_sqrtf(x[e]);
        const uint32_t b = top_bits(x[e]);
        top = top > b ? top : b;
    }
    const uint32_t eb = scale_byte(block_max(top));
    const float inv = scale_inv(eb);
    float y[kQuad];
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        y[e] = x[e] * inv;
        if (ROOT) y[e] = x[e] > 0.0f ? __builtin_fmaxf(y[e], 0x1p-9f) : y[e];
        if ((__float_as_uint(x[e]) & 0x7FFFFFFFu) >= kInfBits) y[e] = __builtin_nanf("");
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
// Workgroup w takes pieces w, w + G, ...; its partial sum goes to memory and
// the last workgroup to finish adds the partials in their order, so the
// result does not depend on which one that is.
constexpr int kSumsqBlock = 256;

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

template <bool GB>
__global__ void __launch_bounds__(kSumsqBlock)
sumsq_kernel(const AdamwTensor *__restrict__ table, const int32_t *__restrict__ map,
             int64_t npieces, int n, double *partial, uint32_t *done, double *out) {
    __shared__ double lds[kSumsqBlock / kWave];
    __shared__ bool last;
    double acc = 0.0;
    for (int64_t piece = blockIdx.x; piece < npieces; piece += gridDim.x) {
        const AdamwTensor &tn = table[map[piece]];
        const int64_t i0 = (piece - tn.piece0) * kAdamwPiece;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t i = i0 + kQuad * (threadIdx.x + h * kSumsqBlock);
            const int64_t left = tn.numel - i;
            if (left <= 0) continue;
            double s[kQuad] = {0.0, 0.0, 0.0, 0.0};
            for (int q = 0; q < n; ++q) {
                float x[kQuad];
                load_quad<GB>(tn.grads[q], i, left, x);
#pragma unroll
                for (int e = 0; e < kQuad; ++e) s[e] += (double)x[e];
            }
#pragma unroll
            for (int e = 0; e < kQuad; ++e) acc = __builtin_fma(s[e], s[e], acc);
        }
    }
    const double s = group_sum(acc, lds);
    if (threadIdx.x == 0) {
        __hip_atomic_store(&partial[blockIdx.x], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        last = __hip_atomic_fetch_add(done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
               gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    double t = 0.0;
    for (unsigned k = threadIdx.x; k < gridDim.x; k += kSumsqBlock)
        t += __hip_atomic_load(&partial[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    t = group_sum(t, lds);
    if (threadIdx.x == 0) {
        *out = t / ((double)n * (double)n);
        __hip_atomic_store(done, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

template <int NR, bool GB, bool PB>
hipError_t launch_typed(const AdamwArgs &a, hipStream_t stream) {
    KernelArgs k = {a.table, a.map, a.n, a.st, a.sc, a.sc_dev, a.ds, a.seed, a.t, a.sumsq,
                    a.max_norm};
    if (a.q8)
        hipLaunchKernelGGL((adamw8_kernel<NR, GB, PB>), dim3((unsigned)a.npieces),
                           dim3(kWave * kPieceWaves), 0, stream, k);
    else
        hipLaunchKernelGGL((adamw32_kernel<NR, GB, PB>), dim3((unsigned)(a.npieces * kPieceWaves)),
                           dim3(kWave), 0, stream, k);
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
    const int64_t want = a.npieces < 1 ? 1 : a.npieces;     // no elements: a sum of zero
    const dim3 g((unsigned)(want < kSumsqGroups ? want : kSumsqGroups)), b(kSumsqBlock);
    if (a.grad_bf16)
        hipLaunchKernelGGL(sumsq_kernel<true>, g, b, 0, stream, a.table, a.map, a.npieces, a.n,
                           a.partial, a.done, a.out);
    else
        hipLaunchKernelGGL(sumsq_kernel<false>, g, b, 0, stream, a.table, a.map, a.npieces, a.n,
                           a.partial, a.done, a.out);
    return hipGetLastError();
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
