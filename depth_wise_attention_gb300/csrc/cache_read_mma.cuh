// cache_read_mma.cuh -- tensor-core read of the quantised depth cache (sm_103a):
//   s_qi = (w_q * g) . v_i / rms_i,  alpha = softmax_i,  o_q = sum_i alpha_qi v_i
// over cache rows (layout: depth_cache.cuh), up to 4 queries.
//
// A warp has one slice, at most 256 channels (16 units of 16) of one head.  A head's
// slices start at a multiple of 4 units, where 16-byte loads are aligned; a slice's
// units outside its head count for nothing: their query values are zero and their
// outputs are not stored, and what they hold is finite (other heads' codes and
// scales; in a stage zeros follow the row's last ones, whose padding is zeros too).  More
// than 16 slices are spread over a cluster of 2, 4 or 8 CTAs (CL): each copies its own
// slices' part of a row, and the warp that forms an item's weights first sends its CTA's
// sums of the dots to the others that have slices of the head (distributed shared
// memory), so that each CTA forms the weights it needs and nothing else is exchanged
// (every warp's dots to every CTA, 32 stores of 4 bytes that each report to one barrier,
// was the pace: 8 FP8 sources, T = 8192, d = 8192 343 us, so 177).
//
// The codes are unpacked straight into mma.sync.m16n8k16 fragments (f16 inputs,
// float accumulation): code * s_b is exact in f16, the row scale 2^k and the
// rms join as factors of a whole row.  The queries and the weights are split into f16
// hi + lo parts (22 significant bits), for bf16 outputs too: with a weight of one f16, off
// by 2^-12 of it, an output much smaller than its terms loses its bits (5% of outputs
// left the bf16 value that they round to; now one in thousands).  The lo parts' MMAs cost 5%
// with FP4 rows (8 sources, T = 32768 269 -> 284 us; 61 sources 255 -> 275 us) and nothing with FP8.
//   pass 1:  D = X Q, X = [16 rows x 16 channels].  The channel order of a dot
//            is free, so a lane's fragments come from the 16-byte pieces that it
//            loads itself; Q (registers, loaded once) has the same order.
//            Columns: query and part (hi, lo).
//   pass 2:  O^T = X^T A, [16 channels x 8 sources] per MMA.  The two halves of
//            k hold the same 8 sources of two channel sets, and A is block-
//            diagonal: columns 0..3 the 4 queries on set one, 4..7 on set two.
//            Lane (g, c) unpacks sources 2c and 2c + 1 of four groups of 8
//            channels (rows g and g + 8 of the two sets), the two sources
//            interleaved before the conversion, so a pair of codes converts at
//            once; MMA j takes the groups' channel j, so a lane ends with 8
//            neighbouring channels of two groups and writes them to global memory
//            itself.  FP4's groups are neighbours: one 16-byte load a row, 32-byte
//            stores, 128 bytes in a line per 8 lanes and 2 queries (with the groups
//            64 channels apart, 16 bytes a lane, the stores took 4 times the L1
//            passes: 363 -> 334 us at T = 32768, d = 4096).
// Source rows arrive by bulk copies in a ring of stages; rows are pitched 16
// bytes past a multiple of 128, which keeps the pieces of pass 1 (two rows, 32
// bytes apart) and of pass 2 (four row pairs) in distinct banks.  The row's sum of
// squares is stored with it, so pass 1 has only dots.
// Items overlap and no CTA barrier stops them: a warp runs pass 1 of item n and
// leaves its partial dots, then runs pass 2 of item n - lag; one warp of the head
// forms item n's weights, needed only after pass 1 of item n + lag (lag is 2 where 5
// stages fit, else 1).  Every hand-over is an mbarrier with a bounded wait.  The warps
// take turns at the weights: with the same warp every time that warp's three jobs set
// the pace (334 -> 304 us; 4 queries, 8 FP4 sources, T = 32768, d = 4096).  Dots and
// weights lie in the item's stage, so its ring is the only counter, and every
// offset of a lane inside a stage is computed once (304 -> 280 us).  With 8 sources HBM and
// the issue of instructions bound the read: of 730 a warp and item (two tokens of 8 FP4 sources) some
// 200 in pass 1 and 260 in pass 2, most of these unpacking.  Past 8 sources nothing is full (61 FP4
// sources: issue slots 58%, ALU pipe 45%, tensor pipe 31%, HBM 26%): one CTA of 16 warps at 128
// registers, of which a few spill (up to 40 bytes), does not hide its latencies; every byte is
// unpacked twice; and with one query three of pass 2's four query columns are zeros.
// Measured with bf16 outputs, 4 queries, d = 4096: 8 FP4 sources, T = 32768, 284 us
// (5.9 TB/s); 8 FP8 sources, T = 32768, 330 us (6.5 TB/s); the same with H = 8, T = 16384,
// 178 us (6.1 TB/s); 61 FP4 sources, T = 4099, 282 us, 1 query 275 (2.2 TB/s).  On clusters,
// d = 8192, T = 8192, 8 FP4 sources 189 us (4.4 TB/s), 8 FP8 sources 182 us (5.9 TB/s).
#pragma once

#include "depth_cache.cuh"

namespace attnres {

constexpr int CM_MAX_WARPS = 16;
constexpr int CM_MAX_STAGES = 8;
constexpr int CM_ROWS = 16;          // rows of a stage: 8 sources of 2 tokens, or 16 sources

constexpr int CM_MAX_CS = 8;         // CTAs of a cluster
constexpr int CM_MAX_HEADS = 64;

// How a row is copied into a stage.  Every copy costs the SM's copy engine about as much as a
// KB of it, so there are as few as the layout allows (three for a FP4 part of a row: T = 8192,
// d = 8192, 8 sources 208 us, two: 181).
enum : int {
    CM_WHOLE = 0,     // as it is
    CM_GAP = 1,       // codes and scales, then the tail behind the zeros that the last slice reads
    CM_PART = 2,      // FP4, a CTA of a cluster: its codes, then everything from the first scale on
    CM_PART_GAP = 3   // a CTA of a cluster: its codes, its scales, and the tail behind zeros
};

struct CacheReadMmaArgs {
    CacheReadArgs r;
    int uh;                          // units per head
    int wph;                         // slices per head
    int nw;                          // warps of a CTA; nw * cs = wph * H
    int cs;                          // CTAs of a cluster
    int16_t ua[CM_MAX_CS], ub[CM_MAX_CS];   // units that each CTA copies; ua a multiple of 16
    int copies;                      // how a row is copied (CM_WHOLE ...)
    uint32_t s_off, t_off;           // where scales and tail begin in a stage's row
    int wpc;                         // floats of a head's partial dots (one per slice, padded)
    int rs;                          // partial dots: floats per value (all heads' or, CL, all warps', padded)
    int nstages;
    int lag;                         // items between pass 1 and pass 2: 1 or 2, nstages >= lag + 2
    uint32_t pitch;                  // bytes between rows of a stage
    uint32_t stage_bytes;
    uint32_t bars;                   // where a stage's barriers begin
    bool wide;                       // out 32-byte aligned
    WaitCfg wait;
};

// A stage holds an item from its copies to its pass 2:
//   rows     16, `pitch` bytes each
//   dots     64 values (K1: token, query, source; K2: row / 8, query, row % 8) of rs
//            floats, wpc per head, one per slice and zeros (CL: one per warp)
//   weights  f16 hi parts (K1 [2 tokens][H][4 queries][8], K2 [H][4][16]), then lo parts
//   factors  K1 units [2 tokens][H][4]; K2 rescaling factors [H][4], final factors [H][4]
//   sums     CL: [2][cs][64], what the CTAs of a head send one another.  A CTA shares at
//            most its first and its last head with others; the first index is 0 for a
//            head that begins in an earlier CTA, 1 for one that begins here
//   barriers the rows have landed; every warp is done with the stage; [H] the head's
//            slices have left their partial dots; [H] the head's weights are there;
//            CL: [2] the sums are there
// with K1 the kernel of at most 8 sources, K2 that of more.
constexpr uint32_t CM_WEIGHT_BYTES = 128, CM_FACTOR_BYTES = 32;     // per head
// (four or more slices: whole float4s, and not a multiple of 32 banks)
inline uint32_t cm_rs(int slices) { return (uint32_t)(slices < 4 ? slices | 1 : (slices + 3) / 4 * 4 + 4); }
inline uint32_t cm_barriers(uint32_t pitch, uint32_t rs, int heads, int cs) {
    return CM_ROWS * pitch + 256 * rs + (2 * CM_WEIGHT_BYTES + CM_FACTOR_BYTES) * (uint32_t)heads + (cs > 1 ? 512 * cs : 0);
}
inline uint32_t cm_stage_bytes(uint32_t pitch, uint32_t rs, int heads, int cs) {
    return (cm_barriers(pitch, rs, heads, cs) + 32 + 16 * (uint32_t)heads + 127) / 128 * 128;
}
// Behind the stages: the abort flag; CL: per head shared with other CTAs (index as in sums) the
// items whose sums this CTA has sent, [2] tokens or halves each, and has armed its barrier for; and
// K2's running state [H][3][4].
constexpr uint32_t CM_SENT = 16, CM_ARMED = 32, CM_STATE = 48;
inline uint32_t cm_aux_bytes(int heads) { return CM_STATE + 48 * (uint32_t)heads; }

// First unit of slice i of a head that begins at unit u0; it and the 15 units after it
// lie in the row where that can be (else the row has zeros behind it in the stage).
__host__ __device__ inline int cm_first_unit(int u0, int i, int units) {
    const int u = (u0 & ~3) + 16 * i, last = units - 16;
    return u > last && last >= 0 && (last & 3) == 0 ? last : u;
}
// The units of slice i that are the head's (u0 to u1) and no earlier slice's.
__host__ __device__ inline uint32_t cm_mask(int u0, int u1, int i, int first) {
    const int from = i == 0 ? u0 : (u0 & ~3) + 16 * i, to = from < u1 ? (first + 16 < u1 ? first + 16 : u1) : from;
    return to > from ? (uint32_t)((1 << (to - first)) - (1 << (from - first))) : 0u;
}
// Slices per head: what the head with the least favourable start needs.
inline int cm_slices(int uh, int H) {
    int most = 0;
    for (int h = 0; h < H; ++h) {
        const int start = h * uh & ~3, n = ((h + 1) * uh - start + 15) / 16;
        if (n > most) most = n;
    }
    return most;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with a zero accumulator.
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t cm_lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t cm_lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float2 cm_lds64f(uint32_t a) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ void cm_sts(uint32_t a, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void cm_sts_h(uint32_t a, float v) {
    const __half h = __float2half_rn(v);
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"(*reinterpret_cast<const uint16_t *>(&h)) : "memory");
}

__device__ __forceinline__ void cm_bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void cm_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// CL: what the barrier stands for was written by other CTAs of the cluster too.
template <bool CL>
__device__ __forceinline__ bool cm_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if constexpr (CL)
        asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
                     " selp.u32 %0, 1, 0, p;\n}\n"
                     : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    else
        asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                     " selp.u32 %0, 1, 0, p;\n}\n"
                     : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ int cm_aborted(uint32_t flag) {
    int v;
    asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(v) : "r"(flag));
    return v;
}
// Raises the abort flag of every CTA of the cluster (this one's alone where there is none): what a
// CTA that gave up would have sent the others never comes, and they must not take anything else for it.
__device__ __forceinline__ void cm_abort(uint32_t flag) {
    uint32_t n;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    for (uint32_t r = 0; r < n; ++r)
        asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n"
                     " st.relaxed.cluster.shared::cluster.u32 [a], %2;\n}\n" ::"r"(flag), "r"(r), "r"(1) : "memory");
}
// mbar_wait_bounded, with 64 tries between looks at the clock: the hand-overs here
// are waited for in every item, and reading the clock takes longer than most waits.
// HEED: give up at once when another warp has.
template <bool CL = false, bool HEED = true>
__device__ __forceinline__ bool cm_wait(uint32_t bar, uint32_t parity, uint32_t flag, const WaitCfg &cfg) {
    uint64_t t0 = 0;
    for (uint32_t n = 0; !cm_try_wait<CL>(bar, parity); ++n)
        if ((n & 63) == 0) {
            if (HEED && cm_aborted(flag)) return false;
            if (n == 0) continue;
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > cfg.timeout_ns) {
                atomicOr(cfg.status, DEV_ERR_TIMEOUT);
                cm_abort(flag);
                return false;
            }
        }
    return true;
}

// First channel (of a slice) that lane column c feeds to k-step s of pass 1:
// channels +0, +1 are k 2c, 2c + 1 and channels +2, +3 are k 2c + 8, 2c + 9.
template <int FMT>
__device__ __forceinline__ int cm_channel(int s, int c) {
    return FMT == CACHE_FP4 ? c * 64 + 4 * s : (s >> 3) * 128 + c * 32 + 4 * (s & 7);
}

// Pass-1 B fragments of a warp's slice: query q = g/2 with the gain folded in,
// its hi part in column 2q, its lo part in column 2q + 1, both scaled by a
// power of two that brings the slice's largest value to [2^13, 2^14): the parts
// then keep 22 bits.  mask: the slice's units inside its head; the others are zeros.
// Returns the inverse of the scale of query c (the query whose dots this lane will hold).
template <int FMT>
__device__ __forceinline__ float cm_query_fragments(const CacheReadArgs &a, int cbase, uint32_t mask, int g, int c,
                                                    uint32_t (&bq)[16][2]) {
    const int q = g >> 1, part = g & 1;
    auto in_head = [&](int s) { return (mask >> (cm_channel<FMT>(s, c) >> 4) & 1) != 0; };
    // (held whole: the fragments' registers are not in use yet, and one round of loads is
    // most of what a launch with few items costs)
    float4 v[16];
    float m = 0.f;
#pragma unroll
    for (int s = 0; s < 16; ++s)
        v[s] = q < a.n_q && in_head(s) ? __ldg(reinterpret_cast<const float4 *>(a.queries + (size_t)q * a.row.d + cbase + cm_channel<FMT>(s, c)))
                         : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < 16; ++s) {
        if (a.gain && in_head(s)) {
            const float4 k = __ldg(reinterpret_cast<const float4 *>(a.gain + cbase + cm_channel<FMT>(s, c)));
            v[s] = make_float4(v[s].x * k.x, v[s].y * k.y, v[s].z * k.z, v[s].w * k.w);
        }
        m = fmaxf(m, fmaxf(fmaxf(fabsf(v[s].x), fabsf(v[s].y)), fmaxf(fabsf(v[s].z), fabsf(v[s].w))));
    }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    int e = (int)(__float_as_uint(m) >> 23) - 127;       // m in [2^e, 2^(e+1))
    e = e < -100 ? -100 : e > 126 ? 126 : e;
    const float sc = __uint_as_float((uint32_t)(127 + 13 - e) << 23);
#pragma unroll
    for (int s = 0; s < 16; ++s) {
        float p[4] = {v[s].x * sc, v[s].y * sc, v[s].z * sc, v[s].w * sc};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float hi = __half2float(__float2half_rn(p[i]));
            p[i] = part == 0 ? hi : p[i] - hi;
        }
        bq[s][0] = pack_h2(p[0], p[1]);
        bq[s][1] = pack_h2(p[2], p[3]);
    }
    const float inv = __uint_as_float((uint32_t)(127 - 13 + e) << 23);
    return __shfl_sync(0xffffffffu, inv, 8 * c);         // lane (g = 2c, 0)
}

// Pass 1 over the 16 rows of a stage: r0, r1 are the shared addresses of this
// lane's slice of rows g and g + 8 (codes), s0, s1 those of its scale bytes.
// dot0 and dot1: rows g and g + 8 against query c.  CH: independent chains of MMAs.
template <int FMT, int CH>
__device__ __forceinline__ void cm_pass1(uint32_t r0, uint32_t r1, uint32_t s0, uint32_t s1,
                                         const uint32_t (&bq)[16][2], float &dot0, float &dot1) {
    float d[CH][4];
#pragma unroll
    for (int u = 0; u < CH; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[u][e] = 0.f;
    if constexpr (FMT == CACHE_FP4) {
        const uint32_t w0 = cm_lds32(s0), w1 = cm_lds32(s1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 c0 = lds128u(r0 + 16 * h), c1 = lds128u(r1 + 16 * h);
            const uint32_t a0[4] = {c0.x, c0.y, c0.z, c0.w}, a1[4] = {c1.x, c1.y, c1.z, c1.w};
            uint32_t f0 = 0, f1 = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if ((w & 1) == 0) {
                    const int b = 2 * h + (w >> 1);
                    f0 = e4m3x2_to_h2(__byte_perm(w0, 0, b * 0x11));
                    f1 = e4m3x2_to_h2(__byte_perm(w1, 0, b * 0x11));
                }
                uint32_t x0[4], x1[4];
                e2m1x8_to_h2(a0[w], x0);
                e2m1x8_to_h2(a1[w], x1);
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    x0[p] = hmul2_u(x0[p], f0);
                    x1[p] = hmul2_u(x1[p], f1);
                }
                const int s = 8 * h + 2 * w;
                mma_f16(d[2 * w % CH], x0[0], x1[0], x0[1], x1[1], bq[s][0], bq[s][1]);
                mma_f16(d[(2 * w + 1) % CH], x0[2], x1[2], x0[3], x1[3], bq[s + 1][0], bq[s + 1][1]);
            }
        }
    } else {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint32_t off = (uint32_t)((b >> 1) * 128 + (b & 1) * 16);
            const uint4 c0 = lds128u(r0 + off), c1 = lds128u(r1 + off);
            const uint32_t a0[4] = {c0.x, c0.y, c0.z, c0.w}, a1[4] = {c1.x, c1.y, c1.z, c1.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t x0[2], x1[2];
                e4m3x4_to_h2(a0[w], x0[0], x0[1]);
                e4m3x4_to_h2(a1[w], x1[0], x1[1]);
                mma_f16(d[w % CH], x0[0], x1[0], x0[1], x1[1], bq[4 * b + w][0], bq[4 * b + w][1]);
            }
        }
    }
#pragma unroll
    for (int u = 1; u < CH; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[0][e] += d[u][e];
    dot0 = d[0][0] + d[0][1];
    dot1 = d[0][2] + d[0][3];
}

// First channel (of a slice) of this lane's group of row r (0: g, 1: g + 8) and set z.
template <int FMT>
__device__ __forceinline__ int cm_group(int g, int z, int r) {
    return FMT == CACHE_FP4 ? 32 * g + 16 * z + 8 * r : 16 * g + 8 * z + 128 * r;
}

// Pass 2 over 8 rows: p0, p1 are the shared addresses of this lane's first group in
// rows 2c and 2c + 1, q0, q1 those of its scale bytes; whi, wlo the
// fragment word of the weights of rows 2c, 2c + 1 and query g & 3, in f16 hi and lo
// parts.  acc[j]: channel j of the groups of set c / 2, row
// 0 (elements 0, 1) and row 1 (elements 2, 3), queries 2c and 2c + 1 mod 4.  FIRST:
// acc is overwritten.
template <int FMT, bool FIRST>
__device__ __forceinline__ void cm_pass2(uint32_t p0, uint32_t p1, uint32_t q0, uint32_t q1, int g, uint32_t whi,
                                         uint32_t wlo, float (&acc)[8][4]) {
    const uint32_t h0 = g < 4 ? whi : 0u, h1 = g < 4 ? 0u : whi;
    const uint32_t l0 = g < 4 ? wlo : 0u, l1 = g < 4 ? 0u : wlo;
    auto step = [&](float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
        if constexpr (FIRST) mma_f16_zero(d, a0, a1, a2, a3, h0, h1);
        else mma_f16(d, a0, a1, a2, a3, h0, h1);
        mma_f16(d, a0, a1, a2, a3, l0, l1);
    };
    if constexpr (FMT == CACHE_FP4) {
        // words 4g .. 4g + 3: (set, row) = (0, 0), (0, 1), (1, 0), (1, 1); one scale per set
        const uint4 u = lds128u(p0), v = lds128u(p1);
        const uint32_t sc = __byte_perm(cm_lds16(q0), cm_lds16(q1), 0x5140);
        uint32_t f[2];
        e4m3x4_to_h2(sc, f[0], f[1]);
        const uint32_t a[4] = {u.x, u.y, u.z, u.w}, b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {
            uint32_t x[4][4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                // channels 0, 2, 4, 6 or 1, 3, 5, 7 of both sources, a byte each
                e2m1x8_to_h2(odd ? ((a[w] >> 4) & 0x0f0f0f0fu) | (b[w] & 0xf0f0f0f0u)
                                 : (a[w] & 0x0f0f0f0fu) | ((b[w] << 4) & 0xf0f0f0f0u), x[w]);
#pragma unroll
                for (int p = 0; p < 4; ++p) x[w][p] = hmul2_u(x[w][p], f[w >> 1]);
            }
#pragma unroll
            for (int p = 0; p < 4; ++p) step(acc[2 * p + odd], x[0][p], x[1][p], x[2][p], x[3][p]);
        }
    } else {
        uint4 u[2], v[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            u[r] = lds128u(p0 + 128 * r);
            v[r] = lds128u(p1 + 128 * r);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t x[4][4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int r = w & 1;
                const uint32_t a = w < 2 ? (half ? u[r].y : u[r].x) : (half ? u[r].w : u[r].z);
                const uint32_t b = w < 2 ? (half ? v[r].y : v[r].x) : (half ? v[r].w : v[r].z);
                e4m3x4_to_h2(__byte_perm(a, b, 0x5140), x[w][0], x[w][1]);
                e4m3x4_to_h2(__byte_perm(a, b, 0x7362), x[w][2], x[w][3]);
            }
#pragma unroll
            for (int p = 0; p < 4; ++p) step(acc[4 * half + p], x[0][p], x[1][p], x[2][p], x[3][p]);
        }
    }
}

// 32 bytes to global memory: one store where they are aligned to 32 (`wide`), else two.
__device__ __forceinline__ void cm_store32(unsigned char *p, bool wide, const uint32_t (&v)[8]) {
    if (wide)
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
    else {
        stg128_cs(p, make_uint4(v[0], v[1], v[2], v[3]));
        stg128_cs(p + 16, make_uint4(v[4], v[5], v[6], v[7]));
    }
}

// Writes a warp's slice of a token, times the units m.x (query q = 2c mod 4) and
// m.y (q + 1), powers of two (POW2).  o: this lane's first channel of query q; qs:
// bytes between queries; nq: queries from q on (0: none of this lane's channels is the
// head's); rows: FP8, which of the lane's two groups are (bits).
template <typename Tout, int FMT, bool POW2>
__device__ __forceinline__ void cm_store(unsigned char *o, int64_t qs, int nq, int rows, bool wide,
                                         const float (&acc)[8][4], float2 m) {
    constexpr int B = Elem<Tout>::BYTES;
    constexpr int ROW = (FMT == CACHE_FP4 ? 8 : 128) * B;     // bytes between a lane's two groups
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (nq <= k) continue;
        const float f = k ? m.y : m.x;
        unsigned char *p = o + k * qs;
        if constexpr (B == 2) {
            uint32_t v[8];
            const uint32_t f2 = f2_to_bf2(f, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = 2 * (j >> 2) + k, c = 2 * (j & 3);
                if constexpr (POW2) {
                    // a power of two: rounded first, scaled in bf16 (exact but for subnormal results)
                    const uint32_t x = f2_to_bf2(acc[c][e], acc[c + 1][e]);
                    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v[j]) : "r"(x), "r"(f2));
                } else {
                    v[j] = f2_to_bf2(acc[c][e] * f, acc[c + 1][e] * f);
                }
            }
            if constexpr (ROW == 16) {
                cm_store32(p, wide, v);
            } else {
                if (rows & 1) stg128_cs(p, make_uint4(v[0], v[1], v[2], v[3]));
                if (rows & 2) stg128_cs(p + ROW, make_uint4(v[4], v[5], v[6], v[7]));
            }
        } else {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                uint32_t v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(acc[j][2 * r + k] * f);
                if (FMT == CACHE_FP4 || (rows >> r & 1)) cm_store32(p + r * ROW, wide, v);
            }
        }
    }
}

// A weight's f16 parts: hi at `a`, lo `lo` bytes further.
__device__ __forceinline__ void cm_put_weight(uint32_t a, uint32_t lo, float w) {
    cm_sts_h(a, w);
    cm_sts_h(a + lo, w - __half2float(__float2half_rn(w)));
}

// The same over n warps' (CL), whole float4s first if they are aligned.
__device__ __forceinline__ float cm_sum_warps(uint32_t p, int n) {
    float s = 0.f;
    int w = 0;
    if ((p & 15) == 0)
#pragma unroll 4
        for (; w + 4 <= n; w += 4) {
            const float4 x = lds128f(p + 4 * w);
            s += (x.x + x.y) + (x.z + x.w);
        }
#pragma unroll 4
    for (; w < n; ++w) s += lds32f(p + 4 * w);
    return s;
}
// Sum over a head's slices of one value's partial dots: up to 3, or whole float4s.
__device__ __forceinline__ float cm_sum(uint32_t p, int wpc) {
    if (wpc < 4) {
        float s = lds32f(p);
        for (int w = 1; w < wpc; ++w) s += lds32f(p + 4 * w);
        return s;
    }
    float4 s = lds128f(p);
#pragma unroll 4
    for (int w = 4; w < wpc; w += 4) {
        const float4 x = lds128f(p + 4 * w);
        s = make_float4(s.x + x.x, s.y + x.y, s.z + x.z, s.w + x.w);
    }
    return (s.x + s.y) + (s.z + s.w);
}

// Score of a row as cache_key_score; the row scale's inverse from its bits (a
// power of two; a marked row's NaN comes back through c - c).
__device__ __forceinline__ float cm_score(float dot, float ss, float inv_dh, float eps, float c) {
    const float ic = __uint_as_float(0x7f000000u - __float_as_uint(c));
    const float ms = fmaf(ss, inv_dh, eps > 0.f ? eps * ic * ic : 0.f);
    return ms == 0.f ? 0.f : dot * rsqrtf(ms) + (c - c);
}

// 2^floor(log2 x) of a positive normal float, and its inverse.
__device__ __forceinline__ float cm_pow2(float x) { return __uint_as_float(__float_as_uint(x) & 0x7f800000u); }
__device__ __forceinline__ float cm_inv_pow2(float p) { return __uint_as_float(0x7f000000u - __float_as_uint(p)); }

// The weights alpha * 2^k of a query are taken in units that bring the largest to
// [2^14, 2^15) where a token has at most 8 sources: it and every weight down to 2^-17 of it is
// kept to 22 bits (its lo part is a normal f16); below that the error is 2^-25 units, 2^-39 of
// the largest weight (a channel in which every heavier source is exactly zero shows it,
// nothing else does).  Past 8 sources the largest weight of a reference starts at 2^8 to 2^9 units
// (cm_form16), so that later ones have room: 22 bits down to 2^-11 of it, then 2^-33 of it.
constexpr float CM_WEIGHT_TOP = 16384.f;

// What a warp works on.
struct CMSlice {
    int rank;                   // CTA in its cluster
    int head, slice;            // slice counts over all heads
    int local, nl;              // this warp among the head's warps in this CTA, and their number
    int chan;                   // first channel
    uint32_t mask;              // its units inside the head
    uint32_t code, scale;       // its offsets in a stage's row
};
template <int FMT, bool CL>
__device__ __forceinline__ CMSlice cm_slice(const CacheReadMmaArgs &a, int warp) {
    CMSlice s;
    s.rank = 0;
    if constexpr (CL) asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(s.rank));
    const int first = s.rank * a.nw;
    s.slice = first + warp;
    s.head = s.slice / a.wph;
    const int h0 = s.head * a.wph, lo = h0 > first ? h0 : first;
    const int hi = h0 + a.wph < first + a.nw ? h0 + a.wph : first + a.nw;
    s.local = s.slice - lo;
    s.nl = hi - lo;
    const int u0 = s.head * a.uh, u1 = u0 + a.uh, ua = a.ua[s.rank];
    int u = cm_first_unit(u0, s.slice - h0, a.r.row.d / 16);
    s.mask = cm_mask(u0, u1, s.slice - h0, u);
    if (s.mask == 0) u = ua;    // (an empty slice goes through the motions on the first units)
    s.chan = 16 * u;
    s.code = (uint32_t)(u - ua) * (FMT == CACHE_FP4 ? 8 : 16);
    s.scale = a.s_off + (a.copies == CM_PART       ? (a.r.row.scale_off & 15) + (uint32_t)u
                         : a.copies == CM_PART_GAP ? (a.r.row.scale_off + (uint32_t)ua & 15) + (uint32_t)(u - ua)
                                                   : (uint32_t)u);
    return s;
}

// Barriers of a CTA whose first slice is `first`.  per_item: warps of a head that write
// its weights of an item, if it has as many here.
__device__ __forceinline__ void cm_init_barriers(const CacheReadMmaArgs &a, uint32_t stage0, uint32_t flag, int first,
                                                 int per_item, int tid, int nthreads) {
    const int H = a.r.row.H;
    for (int i = tid; i < a.nstages * (H + 1); i += nthreads) {
        const int s = i / (H + 1), h = i - s * (H + 1);
        const uint32_t b = stage0 + s * a.stage_bytes + a.bars;
        if (h == H) {
            cm_bar_init(b, 1);
            cm_bar_init(b + 8, a.nw);
            cm_bar_init(b + 16 + 16 * H, 1);
            cm_bar_init(b + 24 + 16 * H, 1);
            continue;
        }
        const int h0 = h * a.wph, lo = h0 > first ? h0 : first;
        const int hi = h0 + a.wph < first + a.nw ? h0 + a.wph : first + a.nw, nl = hi - lo;
        cm_bar_init(b + 16 + 8 * h, nl < 1 ? 1 : nl);
        cm_bar_init(b + 16 + 8 * (H + h), nl < 1 ? 1 : nl < per_item ? nl : per_item);
    }
    if (tid < (int)CM_STATE / 4) asm volatile("st.volatile.shared.s32 [%0], 0;" ::"r"(flag + 4 * tid) : "memory");
    mbar_init_fence();
}

// The copies of one row: whole, or codes, scales and tail apart.
struct CMCopy {
    uint32_t codes, scale_src, scale_dst, scales, tail, total;
};
template <int FMT>
__device__ __forceinline__ CMCopy cm_copy_plan(const CacheReadMmaArgs &a, int rank) {
    CMCopy p = {};
    const uint32_t ua = (uint32_t)a.ua[rank], n = (uint32_t)a.ub[rank] - ua;
    if (a.copies <= CM_GAP) {
        p.codes = a.copies == CM_GAP ? a.r.row.tail_off : a.r.row.bytes;
    } else {
        p.codes = (n * (FMT == CACHE_FP4 ? 8 : 16) + 15) & ~15u;
        if (a.copies == CM_PART) {
            p.scale_src = a.r.row.scale_off & ~15u;
            p.scales = a.r.row.bytes - p.scale_src;
        } else if (FMT == CACHE_FP4 && n != 0) {
            const uint32_t at = a.r.row.scale_off + ua;
            p.scale_src = at & ~15u;
            p.scales = ((at & 15u) + n + 15) & ~15u;
        }
    }
    if (a.copies == CM_GAP || a.copies == CM_PART_GAP) p.tail = a.r.row.bytes - a.r.row.tail_off;
    p.total = p.codes + p.scales + p.tail;
    return p;
}
template <int FMT>
__device__ __forceinline__ void cm_copy_row(const CacheReadMmaArgs &a, const CMCopy &p, int rank, unsigned char *dst,
                                            const unsigned char *row, uint64_t *bar, uint64_t pol) {
    if (p.codes) bulk_g2s(dst, row + (uint32_t)a.ua[rank] * (FMT == CACHE_FP4 ? 8 : 16), p.codes, bar, pol);
    if (p.scales) bulk_g2s(dst + a.s_off, row + p.scale_src, p.scales, bar, pol);
    if (p.tail) bulk_g2s(dst + a.t_off, row + a.r.row.tail_off, p.tail, bar, pol);
}

__device__ __forceinline__ void cm_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Leaves a warp's partial dots of 16 rows at `at` (rows g) and 128 rs further (g + 8).
__device__ __forceinline__ void cm_leave_dots(const CacheReadMmaArgs &a, uint32_t at, uint32_t bar, float dot0, float dot1,
                                              int lane) {
    cm_sts(at, dot0);
    cm_sts(at + 128 * a.rs, dot1);
    __syncwarp();
    if (lane == 0) cm_arrive(bar);
}

// A CTA's share in a head (CL): the head's CTAs, and where their sums are.
struct CMShare {
    int r0, r1, slot;
};
__device__ __forceinline__ void cm_count(uint32_t a, int v) {
    asm volatile("st.volatile.shared.s32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
// Sends this CTA's sum of value 32 k + lane of an item to the head's other CTAs; it reports to their
// barriers when it has landed.  Only a CTA that has not given up does: no warp adds to the sums
// or arrives at a barrier before its turn unless the flag was up first.
__device__ __forceinline__ void cm_send_sum(const CacheReadMmaArgs &a, const CMSlice &s, const CMShare &sh, uint32_t st, int item,
                                            int k, float v, uint32_t flag, int lane) {
    const int H = a.r.row.H;
    if (lane == 0 && sh.r1 > sh.r0) cm_count(flag + CM_SENT + 4 * (2 * sh.slot + k), item + 1);
    for (int r = sh.r0; r <= sh.r1; ++r) {
        if (r == s.rank) continue;
        const int slot = s.head * a.wph < r * a.nw ? 0 : 1;
        uint32_t to, tb;
        asm("mapa.shared::cluster.u32 %0, %1, %2;"
            : "=r"(to) : "r"(st + a.bars - 512 * a.cs + (uint32_t)((slot * a.cs + s.rank) * 64 + 32 * k + lane) * 4), "r"(r));
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(tb) : "r"(st + a.bars + 16 + 16 * H + 8 * slot), "r"(r));
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];"
                     ::"r"(to), "r"(__float_as_uint(v)), "r"(tb) : "memory");
    }
}
// The one arrival of a sums barrier: 64 values from each other CTA of the head.
__device__ __forceinline__ void cm_expect_sums(const CacheReadMmaArgs &a, const CMShare &sh, uint32_t st, int item, uint32_t flag,
                                               int lane) {
    if (lane == 0 && sh.r1 > sh.r0) {
        cm_count(flag + CM_ARMED + 4 * sh.slot, item + 1);
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                     ::"r"(st + a.bars + 16 + 16 * a.r.row.H + 8 * sh.slot), "r"(256 * (sh.r1 - sh.r0)) : "memory");
    }
}
// The head's sum of value 32 k + lane, always in the same order.
__device__ __forceinline__ float cm_all_sums(const CacheReadMmaArgs &a, const CMSlice &s, const CMShare &sh, uint32_t st, int k,
                                             float v, int lane) {
    float sum = 0.f;
    for (int r = sh.r0; r <= sh.r1; ++r)
        sum += r == s.rank ? v : lds32f(st + a.bars - 512 * a.cs + (uint32_t)((sh.slot * a.cs + r) * 64 + 32 * k + lane) * 4);
    return sum;
}

// The end of a cluster: no CTA leaves while another may still write into it.  Where none gave up, each
// has waited for all that was sent to it.  Otherwise (every flag is up then) sums may be on their way:
// of a head's last armed item, or of the one after it, for a CTA sends an item's only when it has
// the others' of the item before.  Their number is what the senders counted, so the barriers of
// these two items are made to complete when they have landed.
__device__ __forceinline__ void cm_leave_cluster(const CacheReadMmaArgs &a, int rank, uint32_t stage0, uint32_t flag, int tid) {
    cm_cluster_sync();
    if (!cm_aborted(flag)) return;
    if (tid == 0)
        for (int slot = 0; slot < 2; ++slot) {
            const int first = rank * a.nw, head = (slot == 0 ? first : first + a.nw - 1) / a.wph, s0 = head * a.wph;
            const int r0 = s0 / a.nw, r1 = (s0 + a.wph - 1) / a.nw;
            if ((s0 < first ? 0 : 1) != slot || r1 == r0) continue;
            const int armed = cm_aborted(flag + CM_ARMED + 4 * slot);
            for (int item = armed > 0 ? armed - 1 : 0; item <= armed; ++item) {
                uint32_t bytes = 0;
                for (int r = r0; r <= r1; ++r)
                    for (int k = 0; k < 2 && r != rank; ++k) {
                        const uint32_t at = flag + CM_SENT + 4 * (2 * (s0 < r * a.nw ? 0 : 1) + k);
                        int sent;
                        asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n"
                                     " ld.relaxed.cluster.shared::cluster.s32 %0, [a];\n}\n"
                                     : "=r"(sent) : "r"(at), "r"(r) : "memory");
                        if (sent > item) bytes += 128;
                    }
                const uint32_t bar = stage0 + item % a.nstages * a.stage_bytes + a.bars + 16 + 16 * a.r.row.H + 8 * slot;
                if (item < armed) {
                    const uint32_t never = 256 * (uint32_t)(r1 - r0) - bytes;
                    if (never)
                        asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(never)
                                     : "memory");
                } else if (bytes) {
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
                } else {
                    continue;
                }
                cm_wait<true, false>(bar, (uint32_t)(item / a.nstages) & 1, flag, a.wait);
            }
        }
    cm_cluster_sync();
}

// A position in the ring of stages.
struct CMRing {
    int s = 0;
    uint32_t par = 0, base;
    __device__ __forceinline__ void next(const CacheReadMmaArgs &a, uint32_t stage0) {
        base += a.stage_bytes;
        if (++s == a.nstages) { s = 0; par ^= 1u; base = stage0; }
    }
};

// The copies of items.  The first nstages items are issued at the start, by warp 0; from
// then on the stage of item it - lag - 1, done with, is refilled at iteration it with the item
// nstages further, by the CTA's warps in turn (always by warp 0, that warp set the pace:
// 8 FP4 sources, T = 32768, d = 4096 292 us, so 272).
struct CMRefill {
    int turn;           // iterations until this warp's next refill
    int last = -1;      // the last item that it issued
    bool on;
    // (a test may stop all copies, 1, or those of the CTA of rank r behind its first items, 2 + r)
    template <typename F>
    __device__ __forceinline__ CMRefill(const CacheReadMmaArgs &a, uint32_t stage0, int rank, int warp, int n_items, const F &issue)
        : turn(warp), on(a.wait.inject_stall == 0 || (a.wait.inject_stall > 1 && a.wait.inject_stall != 2 + rank)) {
        if (warp == 0 && a.wait.inject_stall != 1)
            for (int i = 0; i < n_items && i < a.nstages; ++i) issue(i, stage0 + i * a.stage_bytes);
    }
    // r2: the position of item it - lag
    template <typename F>
    __device__ __forceinline__ void step(const CacheReadMmaArgs &a, int it, int n_items, const CMRing &r2, uint32_t flag,
                                         const F &issue) {
        if (it <= a.lag) return;
        if (--turn >= 0) return;
        turn = a.nw - 1;
        const int item = it - a.lag - 1 + a.nstages;
        if (!on || item >= n_items) return;
        const bool wrap = r2.s == 0;
        const uint32_t base = (wrap ? flag : r2.base) - a.stage_bytes;
        const bool ok = cm_wait(base + a.bars + 8, r2.par ^ (wrap ? 1u : 0u), flag, a.wait);
        on = __all_sync(0xffffffffu, ok);
        if (on) {
            issue(item, base);
            last = item;
        }
    }
    // Copies still in flight after a timeout must land before the CTA exits (without one, every warp
    // has waited for every item).
    __device__ __forceinline__ void drain(const CacheReadMmaArgs &a, uint32_t stage0, int warp, int lane, int n_items,
                                          uint32_t flag) const {
        if (lane != 0 || !cm_aborted(flag)) return;
        for (int i = last; i >= 0 && i > last - a.nstages; i -= a.nw)
            cm_wait<false, false>(stage0 + i % a.nstages * a.stage_bytes + a.bars, (uint32_t)(i / a.nstages) & 1, flag, a.wait);
        if (warp == 0 && a.wait.inject_stall != 1)
            for (int i = 0; i < n_items && i < a.nstages; ++i)
                cm_wait<false, false>(stage0 + i * a.stage_bytes + a.bars, 0, flag, a.wait);
    }
};

// A lane's offsets inside a stage.
template <int FMT>
struct CMLane {
    uint32_t r1, s1;        // pass 1: codes and scale bytes of row g
    uint32_t p2, q2;        // pass 2: codes and scale bytes of row 2c
    uint32_t dot;           // pass 1's partial dot of row g, query c
    int nq, rows;           // outputs: queries from 2c mod 4 on, FP8's groups
    __device__ __forceinline__ CMLane(const CacheReadMmaArgs &a, const CMSlice &s, int g, int c) {
        r1 = (uint32_t)g * a.pitch + s.code + 32 * c;
        s1 = (uint32_t)g * a.pitch + s.scale + 4 * c;
        p2 = (uint32_t)(2 * c) * a.pitch + s.code + 16 * g;
        q2 = (uint32_t)(2 * c) * a.pitch + s.scale + 2 * g;
        const int column = a.cs > 1 ? s.slice - s.rank * a.nw : s.head * a.wpc + s.slice - s.head * a.wph;
        dot = CM_ROWS * a.pitch + (uint32_t)((c * 8 + g) * a.rs + column) * 4;
        rows = (int)((s.mask >> g & 1) | (s.mask >> (g + 8) & 1) << 1);
        nq = (FMT == CACHE_FP4 ? (s.mask >> (2 * g + (c >> 1)) & 1) != 0 : rows != 0) ? a.r.n_q - 2 * (c & 1) : 0;
    }
};

// Weights of token k of an item and a head, at most 8 sources; lane 8 q + i: query q,
// source i.  dt: its dot.  lse: this CTA writes it.
__device__ __forceinline__ void cm_form8(const CacheReadMmaArgs &a, uint32_t st, int k, int head, int64_t t, float dt,
                                         float inv_dh, int lane, bool lse, uint32_t flag) {
    const int q = lane >> 3, i = lane & 7, H = a.r.row.H;
    const bool on = i < a.r.n_src;
    const uint32_t tail = st + (uint32_t)(8 * k + i) * a.pitch + a.t_off, dots = st + CM_ROWS * a.pitch;
    const uint32_t w0 = dots + 256 * a.rs, f0 = w0 + 2 * CM_WEIGHT_BYTES * H;
    const float cs = lds32f(tail), ss = lds32f(tail + 4 + 4 * head);
    const float score = on ? cm_score(dt, ss, inv_dh, a.r.eps, cs) : -INFINITY;
    const float mx = seg_max<8>(score);
    const float e = on ? __expf(score - mx) : 0.f;
    const float sum = seg_sum<8>(e);
    const float w = on ? __fdividef(e, sum) * cs : 0.f;
    const float p2 = cm_pow2(seg_max<8>(w));
    cm_put_weight(w0 + (uint32_t)(((k * H + head) * 4 + q) * 8 + i) * 2, CM_WEIGHT_BYTES * H,
                      w * (cm_inv_pow2(p2) * CM_WEIGHT_TOP));
    if (i == 0) {
        cm_sts(f0 + (uint32_t)((k * H + head) * 4 + q) * 4, p2 * (1.f / CM_WEIGHT_TOP));
        if (lse && q < a.r.n_q && t < a.r.T && !cm_aborted(flag))
            a.r.lse[((int64_t)q * H + head) * a.r.T + t] = mx + __logf(sum);
    }
}

// K1, at most 8 sources: an item is two tokens, whose 8 rows each fill the 16 rows
// of pass 1.  Row 8 k + i of a stage holds source i of token k.
template <typename Tout, int FMT, bool CL>
__global__ void __launch_bounds__(CM_MAX_WARPS * 32, 1) cache_read_mma_kernel(const CacheReadMmaArgs a) {
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int n_src = a.r.n_src, H = a.r.row.H;
    const uint32_t stage0 = smem_u32(smem), flag = stage0 + a.nstages * a.stage_bytes;
    const CMSlice sl = cm_slice<FMT, CL>(a, warp);

    cm_init_barriers(a, stage0, flag, sl.rank * a.nw, 2, tid, blockDim.x);
    // rows of absent sources are never loaded but enter the MMAs (times zero): zeros, not stale
    // bits; so is what lies between the copies of a row
    for (int s = 0; s < a.nstages; ++s)
        for (int row = 0; row < CM_ROWS; ++row)
            if ((row & 7) >= n_src || a.copies != CM_WHOLE)
                for (uint32_t b = tid * 16; b < a.pitch; b += blockDim.x * 16)
                    *reinterpret_cast<uint4 *>(smem + (size_t)s * a.stage_bytes + row * a.pitch + b) = make_uint4(0, 0, 0, 0);
    if (a.wpc != a.wph)             // (the padding of the partial dots)
        for (int s = 0; s < a.nstages; ++s)
            for (uint32_t b = tid * 16; b < 256 * (uint32_t)a.rs; b += blockDim.x * 16)
                *reinterpret_cast<uint4 *>(smem + (size_t)s * a.stage_bytes + CM_ROWS * a.pitch + b) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_shared();
    __syncthreads();
    if constexpr (CL) cm_cluster_sync();

    const int64_t npairs = (a.r.T + 1) / 2;
    const int bid = CL ? blockIdx.x / a.cs : blockIdx.x, gstride = CL ? gridDim.x / a.cs : gridDim.x;
    const int n_items = (int)((npairs - bid + gstride - 1) / gstride);
    const float inv_dh = 1.f / (float)(16 * a.uh);

    // copies: lane 0 arms the stage's mbarrier, lane 8 k + i copies source i of token k
    const uint64_t pol = l2_policy_evict_first();
    auto issue = [&](int item, uint32_t base) {
        const int64_t t0 = 2 * (bid + (int64_t)item * gstride);
        const int ntok = t0 + 1 < a.r.T ? 2 : 1;
        const CMCopy plan = cm_copy_plan<FMT>(a, sl.rank);
        unsigned char *stage = smem + (base - stage0);
        uint64_t *full = reinterpret_cast<uint64_t *>(stage + a.bars);
        if (lane == 0) mbar_arrive_expect_tx(full, plan.total * n_src * ntok);
        __syncwarp();
        const int k = lane >> 3, i = lane & 7;
        if (k < ntok && i < n_src)
            cm_copy_row<FMT>(a, plan, sl.rank, stage + (size_t)lane * a.pitch,
                             a.r.cache + (t0 + k) * a.r.row.bytes + (int64_t)i * a.r.cache_stride_bytes, full, pol);
    };
    CMRefill rf(a, stage0, sl.rank, warp, n_items, issue);

    uint32_t bq[16][2];
    const float qinv = cm_query_fragments<FMT>(a.r, sl.chan, sl.mask, g, c, bq);
    const int head = sl.head;
    const bool lse = a.r.lse && sl.slice - sl.local == head * a.wph;     // the head's first slice is here
    const CMLane<FMT> at(a, sl, g, c);
    const CMShare share = {head * a.wph / a.nw, ((head + 1) * a.wph - 1) / a.nw, head * a.wph < sl.rank * a.nw ? 0 : 1};
    const uint32_t dots_in = a.bars + 16 + 8 * head, weights_in = dots_in + 8 * H;      // the head's barriers
    const uint32_t w0 = CM_ROWS * a.pitch + 256 * a.rs;
    const uint32_t w_at = w0 + (uint32_t)(head * 64 + (g & 3) * 16 + 4 * c);
    // this lane's outputs: query 2c mod 4 on, its groups of set c / 2
    const int q0 = 2 * (c & 1);
    const uint32_t f_at = w0 + (uint32_t)(2 * CM_WEIGHT_BYTES * H + head * 16 + q0 * 4);
    const int64_t tok_bytes = (int64_t)a.r.row.d * Elem<Tout>::BYTES;
    unsigned char *out = a.r.out + q0 * a.r.out_q_stride_bytes + 2 * (int64_t)bid * tok_bytes +
                         (int64_t)(sl.chan + cm_group<FMT>(g, c >> 1, 0)) * Elem<Tout>::BYTES;
    // the last item of an odd T has one token
    const int single = (a.r.T & 1) && bid + (int64_t)(n_items - 1) * gstride == npairs - 1 ? n_items - 1 : -1;
    // the head's warps take turns forming its weights, one a token: warps rot and rot + 1 this item
    const int nl = sl.nl;
    int turn = sl.local;            // 0: forms the weights of the item's first token, 1: of its second

    CMRing r1, r2;                  // of pass 1's item, it, and of pass 2's, it - lag
    r1.base = r2.base = stage0;
    for (int it = 0; it < n_items + a.lag; ++it) {
        rf.step(a, it, n_items, r2, flag, issue);
        if (it < n_items) {
            cm_wait(r1.base + a.bars, r1.par, flag, a.wait);
            const uint32_t x = r1.base + at.r1, y = r1.base + at.s1, dot = r1.base + at.dot;
            float dot0, dot1;
            cm_pass1<FMT, 4>(x, x + 8 * a.pitch, y, y + 8 * a.pitch, bq, dot0, dot1);
            cm_leave_dots(a, dot, r1.base + dots_in, dot0 * qinv, dot1 * qinv, lane);
        }
        if (it >= a.lag) {
            cm_wait(r2.base + weights_in, r2.par, flag, a.wait);
            const bool live = !cm_aborted(flag);
            const uint32_t wa = r2.base + w_at, fa = r2.base + f_at;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (k == 1 && it - a.lag == single) break;
                const uint32_t whi = cm_lds32(wa + 64 * H * k);
                const uint32_t wlo = cm_lds32(wa + 64 * H * k + CM_WEIGHT_BYTES * H);
                const float2 m = cm_lds64f(fa + 16 * H * k);
                float acc[8][4];
                const uint32_t x = r2.base + at.p2 + 8 * k * a.pitch, y = r2.base + at.q2 + 8 * k * a.pitch;
                cm_pass2<FMT, true>(x, x + a.pitch, y, y + a.pitch, g, whi, wlo, acc);
                if (live) cm_store<Tout, FMT, true>(out + k * tok_bytes, a.r.out_q_stride_bytes, at.nq, at.rows, a.wide, acc, m);
            }
            __syncwarp();
            if (lane == 0) cm_arrive(r2.base + a.bars + 8);
            r2.next(a, stage0);
            out += 2 * gstride * tok_bytes;
        }
        if (it < n_items) {
            const bool forms0 = turn == 0, forms1 = turn == (nl > 1 ? 1 : 0);
            if (forms0 || forms1) {
                cm_wait(r1.base + dots_in, r1.par, flag, a.wait);
                const bool send = CL && !__any_sync(0xffffffffu, cm_aborted(flag));
                float dt[2];
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (k == 0 ? forms0 : forms1) {
                        const uint32_t d = r1.base + CM_ROWS * a.pitch + (uint32_t)((k * 32 + lane) * a.rs) * 4;
                        if constexpr (CL) {
                            dt[k] = cm_sum_warps(d + (warp - sl.local) * 4, nl);
                            if (send) cm_send_sum(a, sl, share, r1.base, it, k, dt[k], flag, lane);
                        } else {
                            dt[k] = cm_sum(d + head * a.wpc * 4, a.wpc);
                        }
                    }
                if (send && share.r1 > share.r0) {
                    if (forms0) cm_expect_sums(a, share, r1.base, it, flag, lane);
                    cm_wait<CL>(r1.base + a.bars + 16 + 16 * H + 8 * share.slot, r1.par, flag, a.wait);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (k == 0 ? forms0 : forms1) {
                        if constexpr (CL) dt[k] = cm_all_sums(a, sl, share, r1.base, k, dt[k], lane);
                        cm_form8(a, r1.base, k, head, 2 * (bid + (int64_t)it * gstride) + k, dt[k], inv_dh, lane, lse, flag);
                    }
                __syncwarp();
                if (lane == 0) cm_arrive(r1.base + weights_in);
            }
            if (nl > 1) {
                turn -= 2;
                if (turn < 0) turn += nl;
            }
            r1.next(a, stage0);
        }
    }
    rf.drain(a, stage0, warp, lane, n_items, flag);
    if constexpr (CL) cm_leave_cluster(a, sl.rank, stage0, flag, tid);
}

// Weights of 16 rows (one item) of a token and head, and the factor by which what
// is summed so far is to be rescaled; lane 8 q + i: query q, rows i and 8 + i.  state:
// the token's reference score, sum and unit, 4 queries each.  dt: the dots.
__device__ __forceinline__ void cm_form16(const CacheReadMmaArgs &a, uint32_t st, int head, int64_t t, int chunk, bool last,
                                          const float (&dt)[2], float inv_dh, int lane, bool lse, uint32_t state, uint32_t flag) {
    const int q = lane >> 3, i = lane & 7, H = a.r.row.H;
    const uint32_t tails = st + a.t_off, dots = st + CM_ROWS * a.pitch;
    const uint32_t w0 = dots + 256 * a.rs, f0 = w0 + 2 * CM_WEIGHT_BYTES * H;
    float score[2], cs[2];
    bool on[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t tail = tails + (uint32_t)(8 * k + i) * a.pitch;
        cs[k] = lds32f(tail);
        const float ss = lds32f(tail + 4 + 4 * head);
        on[k] = chunk * CM_ROWS + 8 * k + i < a.r.n_src;
        score[k] = on[k] ? cm_score(dt[k], ss, inv_dh, a.r.eps, cs[k]) : -INFINITY;
    }
    // Weights e^(s - m) c in units u against the reference (m, u) of the items so far, unless one
    // of them passes f16 there, or e^(s - m) itself passes 2^75 (rows of tiny scale: the sum would
    // pass float before a weight passes f16): then the reference moves to this item's largest score and weight,
    // and the sums are rescaled.  The largest weight of a reference starts at 2^8 to 2^9 units, so
    // that is rare (rescaling at every new maximum: 314 us, so: 302; 61 sources, T = 4099).
    // Nothing lies below 2^-110: row scales do not.
    float m = chunk == 0 ? -INFINITY : lds32f(state + 4 * q), u = chunk == 0 ? 0.f : lds32f(state + 32 + 4 * q);
    float l = chunk == 0 ? 0.f : lds32f(state + 16 + 4 * q);
    const float top = seg_max<8>(fmaxf(score[0], score[1]));
    float e0 = on[0] ? __expf(score[0] - m) : 0.f, e1 = on[1] ? __expf(score[1] - m) : 0.f;
    float f = 1.f;
    const float least = u * 0x1p-60f;
    const bool move = chunk == 0 || seg_max<8>(fmaxf(on[0] ? e0 * fmaxf(cs[0], least) : 0.f,
                                                     on[1] ? e1 * fmaxf(cs[1], least) : 0.f)) > 60000.f * u;
    if (__any_sync(0xffffffffu, move)) {
        const float mn = fmaxf(m, top), keep = chunk == 0 ? 0.f : __expf(m - mn);
        const float n0 = on[0] ? __expf(score[0] - mn) : 0.f, n1 = on[1] ? __expf(score[1] - mn) : 0.f;
        const float w = seg_max<8>(fmaxf(on[0] ? n0 * cs[0] : 0.f, on[1] ? n1 * cs[1] : 0.f));
        if (move) {
            f = u * keep;
            u = fmaxf(cm_pow2(fmaxf(f * 256.f, w)), 7.70371978e-34f) * (1.f / 256.f);
            f *= cm_inv_pow2(u);
            l *= keep;
            m = mn;
            e0 = n0;
            e1 = n1;
        }
    }
    l += seg_sum<8>(e0 + e1);
    const float iu = cm_inv_pow2(u);
    const uint32_t w = w0 + (uint32_t)((head * 4 + q) * 16 + i) * 2;
    cm_put_weight(w, CM_WEIGHT_BYTES * H, on[0] ? e0 * cs[0] * iu : 0.f);
    cm_put_weight(w + 16, CM_WEIGHT_BYTES * H, on[1] ? e1 * cs[1] * iu : 0.f);
    __syncwarp();
    if (i == 0) {
        cm_sts(state + 4 * q, m);
        cm_sts(state + 16 + 4 * q, l);
        cm_sts(state + 32 + 4 * q, u);
        const uint32_t fa = f0 + (uint32_t)(head * 4 + q) * 4;
        cm_sts(fa, f);
        if (last) {
            cm_sts(fa + 16 * H, __fdividef(u, l));
            if (lse && q < a.r.n_q && !cm_aborted(flag))
                a.r.lse[((int64_t)q * H + head) * a.r.T + t] = m + __logf(l);
        }
    }
}

// K2, more than 8 sources: an item is 16 sources of one token; the token's items
// follow one another and are folded together by an online softmax.  The
// accumulators stay in registers, in units of a power of two per query; an
// item's factor rescales them when it moves the reference (cm_form16).
template <typename Tout, int FMT, bool CL>
__global__ void __launch_bounds__(CM_MAX_WARPS * 32, 1) cache_read_mma_multi_kernel(const CacheReadMmaArgs a) {
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int n_src = a.r.n_src, H = a.r.row.H, nchunks = (n_src + CM_ROWS - 1) / CM_ROWS;
    const uint32_t stage0 = smem_u32(smem), flag = stage0 + a.nstages * a.stage_bytes;
    const CMSlice sl = cm_slice<FMT, CL>(a, warp);

    cm_init_barriers(a, stage0, flag, sl.rank * a.nw, 1, tid, blockDim.x);
    // rows that are never loaded (one short item a token) must be zeros; so is what lies between the copies of a row
    for (int s = 0; s < a.nstages; ++s)
        for (uint32_t b = tid * 16; b < CM_ROWS * a.pitch; b += blockDim.x * 16)
            *reinterpret_cast<uint4 *>(smem + (size_t)s * a.stage_bytes + b) = make_uint4(0, 0, 0, 0);
    if (a.wpc != a.wph)             // (the padding of the partial dots)
        for (int s = 0; s < a.nstages; ++s)
            for (uint32_t b = tid * 16; b < 256 * (uint32_t)a.rs; b += blockDim.x * 16)
                *reinterpret_cast<uint4 *>(smem + (size_t)s * a.stage_bytes + CM_ROWS * a.pitch + b) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_shared();
    __syncthreads();
    if constexpr (CL) cm_cluster_sync();

    const int bid = CL ? blockIdx.x / a.cs : blockIdx.x, gstride = CL ? gridDim.x / a.cs : gridDim.x;
    const int n_items = (int)((a.r.T - bid + gstride - 1) / gstride) * nchunks;
    const float inv_dh = 1.f / (float)(16 * a.uh);

    const uint64_t pol = l2_policy_evict_first();
    auto issue = [&](int item, uint32_t base) {
        const int tok = item / nchunks, i0 = (item - tok * nchunks) * CM_ROWS;
        const int rows = n_src - i0 < CM_ROWS ? n_src - i0 : CM_ROWS;
        const CMCopy plan = cm_copy_plan<FMT>(a, sl.rank);
        unsigned char *stage = smem + (base - stage0);
        uint64_t *full = reinterpret_cast<uint64_t *>(stage + a.bars);
        // the rows past the last source of a short item count for nothing, but a weight of zero times
        // what an earlier item left there (another token's bytes, NaN codes if it was never
        // written) need not be zero: they repeat the token's last row
        const int copies = nchunks > 1 ? CM_ROWS : rows;
        if (lane == 0) mbar_arrive_expect_tx(full, plan.total * copies);
        __syncwarp();
        if (lane < copies)
            cm_copy_row<FMT>(a, plan, sl.rank, stage + (size_t)lane * a.pitch,
                             a.r.cache + (bid + (int64_t)tok * gstride) * a.r.row.bytes +
                                 (int64_t)(i0 + (lane < rows ? lane : rows - 1)) * a.r.cache_stride_bytes, full, pol);
    };
    CMRefill rf(a, stage0, sl.rank, warp, n_items, issue);

    uint32_t bq[16][2];
    const float qinv = cm_query_fragments<FMT>(a.r, sl.chan, sl.mask, g, c, bq);
    const int head = sl.head;
    const bool lse = a.r.lse && sl.slice - sl.local == head * a.wph;     // the head's first slice is here
    const CMLane<FMT> at(a, sl, g, c);
    const CMShare share = {head * a.wph / a.nw, ((head + 1) * a.wph - 1) / a.nw, head * a.wph < sl.rank * a.nw ? 0 : 1};
    const uint32_t dots_in = a.bars + 16 + 8 * head, weights_in = dots_in + 8 * H;      // the head's barriers
    const uint32_t w0 = CM_ROWS * a.pitch + 256 * a.rs;
    const uint32_t w_at = w0 + (uint32_t)(head * 128 + (g & 3) * 32 + 4 * c);
    const int q0 = 2 * (c & 1);
    const uint32_t f_at = w0 + (uint32_t)(2 * CM_WEIGHT_BYTES * H + head * 16 + q0 * 4);
    const int64_t tok_bytes = (int64_t)a.r.row.d * Elem<Tout>::BYTES;
    unsigned char *out = a.r.out + q0 * a.r.out_q_stride_bytes + (int64_t)bid * tok_bytes +
                         (int64_t)(sl.chan + cm_group<FMT>(g, c >> 1, 0)) * Elem<Tout>::BYTES;
    // the head's warps take turns forming its weights, an item each
    const int nl = sl.nl;
    int turn = sl.local;

    CMRing r1, r2;
    r1.base = r2.base = stage0;
    int chunk = 0, chunk_p = 0;
    int64_t t = bid;
    float acc[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
    for (int it = 0; it < n_items + a.lag; ++it) {
        rf.step(a, it, n_items, r2, flag, issue);
        if (it < n_items) {
            cm_wait(r1.base + a.bars, r1.par, flag, a.wait);
            const uint32_t x = r1.base + at.r1, y = r1.base + at.s1, dot = r1.base + at.dot;
            float dot0, dot1;
            cm_pass1<FMT, 2>(x, x + 8 * a.pitch, y, y + 8 * a.pitch, bq, dot0, dot1);
            cm_leave_dots(a, dot, r1.base + dots_in, dot0 * qinv, dot1 * qinv, lane);
        }
        if (it >= a.lag) {
            cm_wait(r2.base + weights_in, r2.par, flag, a.wait);
            const uint32_t wa = r2.base + w_at, fa = r2.base + f_at;
            if (chunk_p != 0) {
                const float2 f = cm_lds64f(fa);
                if (f.x != 1.f || f.y != 1.f)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[j][e] *= (e & 1) ? f.y : f.x;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t whi = cm_lds32(wa + 16 * k), wlo = cm_lds32(wa + 16 * k + CM_WEIGHT_BYTES * H);
                const uint32_t x = r2.base + at.p2 + 8 * k * a.pitch, y = r2.base + at.q2 + 8 * k * a.pitch;
                cm_pass2<FMT, false>(x, x + a.pitch, y, y + a.pitch, g, whi, wlo, acc);
            }
            if (++chunk_p == nchunks) {
                if (!cm_aborted(flag))
                    cm_store<Tout, FMT, false>(out, a.r.out_q_stride_bytes, at.nq, at.rows, a.wide, acc, cm_lds64f(fa + 16 * H));
                out += gstride * tok_bytes;
                chunk_p = 0;
            }
            __syncwarp();
            if (lane == 0) cm_arrive(r2.base + a.bars + 8);
            r2.next(a, stage0);
        }
        if (it < n_items) {
            if (turn == 0) {
                // the running state is what the previous item's warp left
                if (chunk != 0 && nl > 1) {
                    const bool wrap = r1.s == 0;
                    cm_wait((wrap ? flag : r1.base) - a.stage_bytes + weights_in, r1.par ^ (wrap ? 1u : 0u), flag, a.wait);
                }
                cm_wait(r1.base + dots_in, r1.par, flag, a.wait);
                const bool send = CL && !__any_sync(0xffffffffu, cm_aborted(flag));
                float dt[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t d = r1.base + CM_ROWS * a.pitch + (uint32_t)((k * 32 + lane) * a.rs) * 4;
                    if constexpr (CL) {
                        dt[k] = cm_sum_warps(d + (warp - sl.local) * 4, nl);
                        if (send) cm_send_sum(a, sl, share, r1.base, it, k, dt[k], flag, lane);
                    } else {
                        dt[k] = cm_sum(d + head * a.wpc * 4, a.wpc);
                    }
                }
                if constexpr (CL) {
                    if (send && share.r1 > share.r0) {
                        cm_expect_sums(a, share, r1.base, it, flag, lane);
                        cm_wait<CL>(r1.base + a.bars + 16 + 16 * H + 8 * share.slot, r1.par, flag, a.wait);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) dt[k] = cm_all_sums(a, sl, share, r1.base, k, dt[k], lane);
                }
                cm_form16(a, r1.base, head, t, chunk, chunk == nchunks - 1, dt, inv_dh, lane, lse, flag + CM_STATE + 48 * head,
                              flag);
                __syncwarp();
                if (lane == 0) cm_arrive(r1.base + weights_in);
            }
            if (--turn < 0) turn = nl - 1;
            if (++chunk == nchunks) { chunk = 0; t += gstride; }
            r1.next(a, stage0);
        }
    }
    rf.drain(a, stage0, warp, lane, n_items, flag);
    if constexpr (CL) cm_leave_cluster(a, sl.rank, stage0, flag, tid);
}

}  // namespace attnres
