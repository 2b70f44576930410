// depth_cache.cu -- writing the quantised depth cache and reading rows back
// (layout: depth_cache.cuh), and the general read of it.
#include "depth_cache.cuh"
#include "dispatch.h"

namespace attnres {

constexpr int CACHE_THREADS = 256;

__device__ __forceinline__ uint32_t add_bf2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// 32 bytes: one load where they are aligned to 32 (`wide`), else two.
__device__ __forceinline__ void ldg32(const unsigned char *p, bool wide, uint32_t *v) {
    if (wide) {
        asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "l"(p));
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p)), b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}
__device__ __forceinline__ void stg32(unsigned char *p, bool wide, const uint32_t *v) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
    } else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// Row scale 2^k: the least k >= CACHE_MIN_EXP with amax <= 2688 * 2^k (FP4: the
// largest code 6 times the largest block scale 448) or 448 * 2^k (FP8), from
// amax's bits: 2688 = 1.3125 * 2^11, 448 = 1.75 * 2^8.
template <int FMT>
__device__ __forceinline__ int row_exponent(uint32_t u) {
    constexpr uint32_t M = FMT == CACHE_FP4 ? 0x280000u : 0x600000u;
    constexpr int E = FMT == CACHE_FP4 ? 11 : 8;
    const int k = (int)(u >> 23) - 127 - E + ((u & 0x7fffffu) > M ? 1 : 0);
    return k > CACHE_MIN_EXP ? k : CACHE_MIN_EXP;
}

// Byte of the least e4m3 value s with 6 s >= a (a <= 2688).  6 s is exact in
// float, so the test decides whatever a / 6 was rounded to; consecutive bytes
// are consecutive values.
__device__ __forceinline__ uint32_t block_scale(float a, float &s) {
    uint16_t b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(0.f), "f"(a * (1.f / 6.f)));
    uint32_t c = b & 0xffu;
    s = h2_to_f2(e4m3x2_to_h2(c)).x;
    if (6.f * s < a) {
        ++c;
        s = h2_to_f2(e4m3x2_to_h2(c)).x;
    }
    return c;
}

// Sixteen channels (one unit) in registers, as stored: 8 words of bf16 pairs or 16 floats.
template <typename T> struct Unit {
    static constexpr int NW = 8 * Elem<T>::BYTES / 2;
    uint32_t w[NW];
    __device__ __forceinline__ void load(const unsigned char *p, bool wide) {
#pragma unroll
        for (int k = 0; k < NW; k += 8) ldg32(p + 4 * k, wide, w + k);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int k = 0; k < NW; ++k) w[k] = 0;
    }
    // The sum rounded to T.  A packed bf16 addition rounds the exact sum once, as a float
    // addition and a rounding to bf16 do: a float sum of two bf16 is inexact only if their
    // exponents are 17 or more apart, far from a border of bf16.
    __device__ __forceinline__ void add(const Unit &o) {
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            if constexpr (Elem<T>::BYTES == 2) w[k] = add_bf2(w[k], o.w[k]);
            else w[k] = __float_as_uint(__uint_as_float(w[k]) + __uint_as_float(o.w[k]));
        }
    }
    // Largest magnitude as its float's bits: those of non-negative floats order as they do,
    // a NaN's above all.
    __device__ __forceinline__ uint32_t amax() const {
        if constexpr (Elem<T>::BYTES == 2) {
            uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
            for (int k = 1; k < NW; ++k) m = __vmaxu2(m, w[k] & 0x7fff7fffu);
            return max(m << 16, m & 0xffff0000u);
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < NW; ++k) m = max(m, w[k] & 0x7fffffffu);
            return m;
        }
    }
    __device__ __forceinline__ float2 pair(int p) const {
        if constexpr (Elem<T>::BYTES == 2) return bf2_to_f2(w[p]);
        else return make_float2(__uint_as_float(w[2 * p]), __uint_as_float(w[2 * p + 1]));
    }
};

// Four pairs of quotients -> a word of e2m1 codes, first pair in the low byte.
__device__ __forceinline__ uint32_t e2m1x8(float2 a, float2 b, float2 c, float2 d) {
    uint32_t w;
    asm("{\n .reg .b8 b0, b1, b2, b3;\n cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n mov.b32 %0, {b0, b1, b2, b3};\n}"
        : "=r"(w)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
    return w;
}

// f32 quotients: v is the correctly rounded quotient, negated, and res the quotient's residual.  If
// it is not exact, its last bit is made odd in the residual's direction; borders are even, so it
// neither stays on one nor reaches one.
__device__ __forceinline__ float odd_quotient(float v, float res) {
    const uint32_t b = __float_as_uint(v);
    if (res == 0.f || (b & 1u) || (b << 1) == 0u) return v;
    return __uint_as_float(((__float_as_uint(res) ^ b) >> 31) ? b + 1u : b - 1u);
}

// Codes of a unit (FP4 with block scale s, S = s 2^k; FP8 with inv = 2^-k), written to p;
// returns the sum of squares of code * s.
//
// FP4 codes are the nearest ones, ties to the even code, of the exact quotient x / S.  A
// product with 1 / S and a residual step round it correctly; its borders have 3 bits, times
// s's 4, so a quotient on a border is exactly that.  One that only rounds to a border is
// impossible for bf16 sources (8 bits against 7: at least 2^-8 of it away); for f32 sources
// the quotient is made odd where it is inexact.  Quotients are formed with their signs turned round:
// where x is -0 (or +0) the product with -1 / S is +0 (-0) and the residual +0, which times -1 / S
// leaves that sign in the sum; added as it is to a product of -0 it would not.
template <typename Tin, int FMT>
__device__ __forceinline__ float unit_codes(const Unit<Tin> &x, unsigned char *p, float s, float S, float inv) {
    if constexpr (FMT == CACHE_FP4) {
        const float R = S > 0.f ? (Elem<Tin>::BYTES == 2 ? __fdividef(1.f, s) * inv : 1.f / s * inv) : 0.f;
        const float2 nR = make_float2(-R, -R), S2 = make_float2(S, S);
        float2 q[8];
        uint32_t low = 1;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 v = x.pair(k), a = fmul2(v, nR);
            q[k] = ffma2(ffma2(a, S2, v), nR, a);
            if constexpr (Elem<Tin>::BYTES == 4)
                low = min(low, min(__float_as_uint(q[k].x) & 0x1fffffu, __float_as_uint(q[k].y) & 0x1fffffu));
        }
        if (Elem<Tin>::BYTES == 4 && low == 0) {
            // some quotient has no more than the 3 bits of a border
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 e = ffma2(q[k], S2, x.pair(k));
                q[k] = make_float2(odd_quotient(q[k].x, e.x), odd_quotient(q[k].y, e.y));
            }
        }
        uint32_t w[2] = {e2m1x8(q[0], q[1], q[2], q[3]) ^ 0x88888888u, e2m1x8(q[4], q[5], q[6], q[7]) ^ 0x88888888u};
        __half2 sq = __float2half2_rn(0.f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // squares of codes: multiples of 1/4, eight of them at most 288 a half: exact in f16
            uint32_t c[4];
            e2m1x8_to_h2(w[h], c);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                sq = __hfma2(*reinterpret_cast<const __half2 *>(&c[k]), *reinterpret_cast<const __half2 *>(&c[k]), sq);
        }
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        const float2 f = __half22float2(sq);
        return (f.x + f.y) * s * s;
    } else {
        const float2 i2 = make_float2(inv, inv);
        uint32_t w[4];
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 y0 = fmul2(x.pair(2 * k), i2), y1 = fmul2(x.pair(2 * k + 1), i2);
            uint16_t c0, c1;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c0) : "f"(y0.y), "f"(y0.x));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c1) : "f"(y1.y), "f"(y1.x));
            w[k] = (uint32_t)c0 | (uint32_t)c1 << 16;
            uint32_t h0, h1;
            e4m3x4_to_h2(w[k], h0, h1);
            const float2 v0 = h2_to_f2(h0), v1 = h2_to_f2(h1);
            acc = ffma2(v0, v0, acc);
            acc = ffma2(v1, v1, acc);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        return acc.x + acc.y;
    }
}

// Quantises rows as they are written.  One row per tpr threads, one unit of 16 channels (one
// block scale) per thread and step; the row stays in registers between the row maximum and
// the codes, so it is read once, and the next row's loads are in flight meanwhile.  bf16 rows
// take two units a thread where they have them: much of a row's work goes by threads.  One
// CTA barrier a row: the sums of squares and the row's tail are finished behind the next row's.
// Memory: 2 or 4 bytes a channel in (twice with f), 0.5625 or 1 out.  Partial + output, bf16
// -> FP4, 32768 x 4096: 163 us with a CTA per row and two barriers, 92 (floor 90).
// Registers are the limit of the CTAs per SM: words of a thread's units, twice with f.  A CTA has
// whole rows' threads (at most CACHE_THREADS), so no warp idles: f32 -> FP4, 12297 x 1056 27.0 ->
// 23.9 us (22.6 now; 32768 x 4096 123, floor 90: the exact quotients of every channel).
template <typename Tin, int FMT, int UPT, bool ADD>
__global__ void __launch_bounds__(CACHE_THREADS, UPT * Elem<Tin>::BYTES <= 2 ? 4 : UPT * Elem<Tin>::BYTES <= 4 ? (ADD ? 2 : 3) : 1)
    cache_quant_kernel(const CacheQuantArgs a) {
    __shared__ uint32_t red[2][CACHE_THREADS / 32];
    __shared__ float uss[2][CACHE_THREADS * UPT];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = tid / a.tpr, tr = tid - r * a.tpr;      // row of the CTA, thread of the row
    const int nwr = a.tpr >> 5, wr = warp - r * nwr;      // warps of a row, warp of the row
    const int rpb = blockDim.x / a.tpr, uph = a.units / a.row.H;
    const int64_t rows = a.n_src * a.T, step = (int64_t)gridDim.x * rpb;
    const uint32_t codes_end = FMT == CACHE_FP4 ? a.row.scale_off + (uint32_t)a.units : a.row.scale_off;
    const float nan = __int_as_float(0x7fffffff);

    // row number and its source and token, step by step
    // (a warp that no row of the CTA needs, r >= rpb, would have none)
    int64_t row = r < rpb ? (int64_t)blockIdx.x * rpb + r : rows, i = row / a.T, t = row - i * a.T;
    const int64_t di = step / a.T, dt = step - di * a.T;
    Unit<Tin> x[UPT], f[ADD ? UPT : 1];
    auto load = [&](int64_t row_, int64_t i_, int64_t t_) {
        const int64_t at = i_ * a.src_stride_bytes + t_ * a.row.d * Elem<Tin>::BYTES;
#pragma unroll
        for (int k = 0; k < UPT; ++k) {
            const int u = k * a.tpr + tr;
            if (row_ < rows && u < a.units) {
                x[k].load(a.src + at + (int64_t)u * 16 * Elem<Tin>::BYTES, a.wide);
                if constexpr (ADD) f[k].load(a.f + at + (int64_t)u * 16 * Elem<Tin>::BYTES, a.wide);
            } else {
                x[k].zero();
                if constexpr (ADD) f[k].zero();
            }
        }
    };
    // the tail of a row whose unit sums are in uss[b]: row scale, sums of squares, padding
    auto tail = [&](int b, unsigned char *p, float scale) {
        for (int h = wr; h < a.row.H; h += nwr) {
            float s = 0.f;
            for (int u = lane; u < uph; u += 32) s += uss[b][r * a.tpr * UPT + h * uph + u];
            s = seg_sum<32>(s);
            if (lane == 0) *reinterpret_cast<float *>(p + a.row.tail_off + 4 + 4 * h) = scale == scale ? s : nan;
        }
        if (wr == nwr - 1) {
            if (lane == 0) *reinterpret_cast<float *>(p + a.row.tail_off) = scale;
            for (uint32_t c = codes_end + lane; c < a.row.tail_off; c += 32) p[c] = 0;
            for (uint32_t c = a.row.tail_off + 4 + 4 * a.row.H + lane; c < a.row.bytes; c += 32) p[c] = 0;
        }
    };
    load(row, i, t);
    int b = 0;
    unsigned char *last = nullptr;
    float last_scale = 0.f;
    for (int64_t base = (int64_t)blockIdx.x * rpb; base < rows; base += step, b ^= 1) {
        const bool ok = row < rows;
        unsigned char *p = a.cache + i * a.cache_stride_bytes + t * a.row.bytes;
        Unit<Tin> v[UPT];
        uint32_t amax = 0, bmax[UPT];
#pragma unroll
        for (int k = 0; k < UPT; ++k) {
            v[k] = x[k];
            if constexpr (ADD) v[k].add(f[k]);        // the block representation: the sum in the sources' type
            bmax[k] = v[k].amax();
            amax = max(amax, bmax[k]);
        }
        row += step;
        i += di;
        t += dt;
        if (t >= a.T) { t -= a.T; ++i; }
        load(row, i, t);
        amax = __reduce_max_sync(0xffffffffu, amax);
        if (lane == 0) red[b][warp] = amax;
        __syncthreads();
        amax = __reduce_max_sync(0xffffffffu, lane < nwr && r < rpb ? red[b][r * nwr + lane] : 0u);
        if (last) tail(b ^ 1, last, last_scale);
        // a row with a NaN, an infinity or a value from 2^126 on reads back as NaN
        const bool bad = amax >= 0x7e800000u;
        const int k2 = row_exponent<FMT>(bad ? 0u : amax);
        const float inv = bad ? 0.f : __uint_as_float((uint32_t)(127 - k2) << 23);
        const float scale = __uint_as_float((uint32_t)(127 + k2) << 23);
#pragma unroll
        for (int k = 0; k < UPT; ++k) {
            const int u = k * a.tpr + tr;
            float ss = 0.f;
            if (ok && u < a.units) {
                if (bad) v[k].zero();
                float s = 0.f;
                if constexpr (FMT == CACHE_FP4)
                    p[a.row.scale_off + u] = (unsigned char)(bad ? 0u : block_scale(__uint_as_float(bmax[k]) * inv, s));
                ss = unit_codes<Tin, FMT>(v[k], p + (size_t)u * (FMT == CACHE_FP4 ? 8 : 16), s, s * scale, inv);
            }
            if (r < rpb) uss[b][r * a.tpr * UPT + u] = ss;
        }
        last = ok ? p : nullptr;
        last_scale = bad ? nan : scale;
    }
    __syncthreads();
    if (last) tail(b ^ 1, last, last_scale);
}

// Reads cache rows back: value = code * s_b * 2^k, exact in float; bf16 values (at most 6
// significant bits) are exact too.  HBM-bound: one unit per thread and step, the loads of two
// units of a row in flight where a thread has as many, other rows' in the SM's other CTAs.  FP4 ->
// bf16, 32768 x 4096: 66 us with a row per CTA, 57 with persistent ones (floor 50).
template <typename Tout, int FMT>
__global__ void __launch_bounds__(CACHE_THREADS) cache_dequant_kernel(const CacheDequantArgs a) {
    using E = Elem<Tout>;
    const int r = threadIdx.x / a.tpr, tr = threadIdx.x - r * a.tpr, rpb = blockDim.x / a.tpr;
    const int64_t rows = a.n_src * a.T, step = (int64_t)gridDim.x * rpb;
    const int64_t di = step / a.T, dt = step - di * a.T;
    constexpr int NP = E::EPV / 2, NW = 8 * E::BYTES / 2;
    if (r >= rpb) return;
    int64_t row = (int64_t)blockIdx.x * rpb + r, i = row / a.T, t = row - i * a.T;
    for (; row < rows;) {
        const unsigned char *p = a.cache + i * a.cache_stride_bytes + t * a.row.bytes;
        unsigned char *out = a.out + i * a.out_stride_bytes + t * a.row.d * E::BYTES;
        const float c = __ldg(reinterpret_cast<const float *>(p + a.row.tail_off));
        const float2 c2 = make_float2(c, c);
#pragma unroll 2
        for (int u = tr; u < a.units; u += a.tpr) {
            uint32_t x[8], v[NW];
            cache_unit_h2<FMT>(p, a.row, u, x);
#pragma unroll
            for (int k = 0; k < NW; k += 4) {
                float2 y[NP];
#pragma unroll
                for (int j = 0; j < NP; ++j) y[j] = fmul2(h2_to_f2(x[k / 4 * NP + j]), c2);
                const uint4 w = E::pack(y);
                v[k] = w.x; v[k + 1] = w.y; v[k + 2] = w.z; v[k + 3] = w.w;
            }
#pragma unroll
            for (int k = 0; k < NW; k += 8) stg32(out + (size_t)u * 16 * E::BYTES + 4 * k, a.wide, v + k);
        }
        row += step;
        i += di;
        t += dt;
        if (t >= a.T) { t -= a.T; ++i; }
    }
}

// The general depth read of a quantised cache: any widths, heads, sources and
// up to 8 queries, one token per CTA.  Scores first (one warp per source and
// head), the softmax over the sources in shared memory, then the weighted sum
// in a second pass over the token's rows (in L1 or L2 by then).
template <typename Tout, int FMT, int NQ>
__global__ void __launch_bounds__(CACHE_THREADS) cache_read_kernel(const CacheReadArgs a) {
    using E = Elem<Tout>;
    extern __shared__ float sc[];   // [n_q][H][n_src] scores, then alpha * row scale
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t t = blockIdx.x;
    const int d = a.row.d, H = a.row.H, units = d / 16, uph = units / H;
    const unsigned char *tok = a.cache + t * a.row.bytes;

    for (int p = warp; p < a.n_src * H; p += CACHE_THREADS / 32) {
        const int i = p / H, h = p - i * H;
        const unsigned char *row = tok + (int64_t)i * a.cache_stride_bytes;
        float2 dot[NQ];
#pragma unroll
        for (int q = 0; q < NQ; ++q) dot[q] = make_float2(0.f, 0.f);
        for (int u = h * uph + lane; u < (h + 1) * uph; u += 32) {
            uint32_t xh[8];
            cache_unit_h2<FMT>(row, a.row, u, xh);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                float2 x0 = h2_to_f2(xh[2 * v]), x1 = h2_to_f2(xh[2 * v + 1]);
                if (a.gain) {
                    const float4 g = __ldg(reinterpret_cast<const float4 *>(a.gain + u * 16 + 4 * v));
                    x0 = fmul2(x0, make_float2(g.x, g.y));
                    x1 = fmul2(x1, make_float2(g.z, g.w));
                }
#pragma unroll
                for (int q = 0; q < NQ; ++q)
                    if (q < a.n_q) {
                        const float4 w = __ldg(reinterpret_cast<const float4 *>(a.queries + (size_t)q * d + u * 16 + 4 * v));
                        dot[q] = ffma2(x0, make_float2(w.x, w.y), dot[q]);
                        dot[q] = ffma2(x1, make_float2(w.z, w.w), dot[q]);
                    }
            }
        }
        const float *tail = reinterpret_cast<const float *>(row + a.row.tail_off);
        const float c = __ldg(tail), ss = __ldg(tail + 1 + h);
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const float s = seg_sum<32>(dot[q].x + dot[q].y);
            if (lane == 0 && q < a.n_q)
                sc[(q * H + h) * a.n_src + i] = cache_key_score(s, ss, 1.f / (float)(d / H), a.eps, c);
        }
    }
    __syncthreads();
    for (int p = warp; p < a.n_q * H; p += CACHE_THREADS / 32) {
        float *s = sc + (size_t)p * a.n_src;
        float m = -INFINITY;
        for (int i = lane; i < a.n_src; i += 32) m = fmaxf(m, s[i]);
        m = seg_max<32>(m);
        float l = 0.f;
        for (int i = lane; i < a.n_src; i += 32) l += __expf(s[i] - m);
        l = seg_sum<32>(l);
        const float inv = 1.f / l;
        for (int i = lane; i < a.n_src; i += 32)
            s[i] = __expf(s[i] - m) * inv *
                   __ldg(reinterpret_cast<const float *>(tok + (int64_t)i * a.cache_stride_bytes + a.row.tail_off));
        if (lane == 0 && a.lse) a.lse[(int64_t)p * a.T + t] = m + __logf(l);
    }
    __syncthreads();
    constexpr int NV = 16 / E::EPV, NP = E::EPV / 2;
    for (int u = tid; u < units; u += CACHE_THREADS) {
        float2 acc[NQ][8];
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int p = 0; p < 8; ++p) acc[q][p] = make_float2(0.f, 0.f);
        const int h = u / uph;
        for (int i = 0; i < a.n_src; ++i) {
            uint32_t xh[8];
            cache_unit_h2<FMT>(tok + (int64_t)i * a.cache_stride_bytes, a.row, u, xh);
            float2 w[NQ];
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const float v = q < a.n_q ? sc[(q * H + h) * a.n_src + i] : 0.f;
                w[q] = make_float2(v, v);
            }
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const float2 x = h2_to_f2(xh[p]);
#pragma unroll
                for (int q = 0; q < NQ; ++q) acc[q][p] = ffma2(x, w[q], acc[q][p]);
            }
        }
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            if (q < a.n_q) {
                uint4 *o = reinterpret_cast<uint4 *>(a.out + q * a.out_q_stride_bytes + t * d * E::BYTES);
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    float2 y[NP];
#pragma unroll
                    for (int j = 0; j < NP; ++j) y[j] = acc[q][v * NP + j];
                    o[(size_t)u * NV + v] = E::pack(y);
                }
            }
    }
}

template <typename T, int FMT, bool ADD>
static bool quant_lookup(int upt, KernelRef *out) {
    switch (upt) {
        case 1: out->fn = reinterpret_cast<const void *>(&cache_quant_kernel<T, FMT, 1, ADD>); return true;
        case 2: out->fn = reinterpret_cast<const void *>(&cache_quant_kernel<T, FMT, 2, ADD>); return true;
        case 4: out->fn = reinterpret_cast<const void *>(&cache_quant_kernel<T, FMT, 4, ADD>); return true;
    }
    return false;
}
template <typename T>
static bool quant_fmt(int fmt, int upt, bool add, KernelRef *out) {
    if (fmt == CACHE_FP4) return add ? quant_lookup<T, CACHE_FP4, true>(upt, out) : quant_lookup<T, CACHE_FP4, false>(upt, out);
    return add ? quant_lookup<T, CACHE_FP8, true>(upt, out) : quant_lookup<T, CACHE_FP8, false>(upt, out);
}

bool lookup_cache_quant(int dt, int fmt, int upt, bool add, KernelRef *out) {
    return dt == 1 ? quant_fmt<__nv_bfloat16>(fmt, upt, add, out) : quant_fmt<float>(fmt, upt, add, out);
}

bool lookup_cache_dequant(int dt, int fmt, KernelRef *out) {
    out->fn = dt == 1 ? (fmt == CACHE_FP4 ? reinterpret_cast<const void *>(&cache_dequant_kernel<__nv_bfloat16, CACHE_FP4>)
                                          : reinterpret_cast<const void *>(&cache_dequant_kernel<__nv_bfloat16, CACHE_FP8>))
                      : (fmt == CACHE_FP4 ? reinterpret_cast<const void *>(&cache_dequant_kernel<float, CACHE_FP4>)
                                          : reinterpret_cast<const void *>(&cache_dequant_kernel<float, CACHE_FP8>));
    return true;
}

template <typename T, int FMT>
static bool read_lookup(int nq, KernelRef *out) {
    switch (nq) {
        case 1: out->fn = reinterpret_cast<const void *>(&cache_read_kernel<T, FMT, 1>); return true;
        case 2: out->fn = reinterpret_cast<const void *>(&cache_read_kernel<T, FMT, 2>); return true;
        case 4: out->fn = reinterpret_cast<const void *>(&cache_read_kernel<T, FMT, 4>); return true;
        case 8: out->fn = reinterpret_cast<const void *>(&cache_read_kernel<T, FMT, 8>); return true;
    }
    return false;
}

bool lookup_cache_read(int dt, int fmt, int nq, KernelRef *out) {
    if (dt == 1) return fmt == CACHE_FP4 ? read_lookup<__nv_bfloat16, CACHE_FP4>(nq, out)
                                         : read_lookup<__nv_bfloat16, CACHE_FP8>(nq, out);
    return fmt == CACHE_FP4 ? read_lookup<float, CACHE_FP4>(nq, out) : read_lookup<float, CACHE_FP8>(nq, out);
}

}  // namespace attnres
