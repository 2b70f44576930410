// cache_read_few.cu -- read of the quantised depth cache for few tokens (sm_103a).
//
// A decoded token is a few KB of cache rows and its read is all latency, so a token is
// spread over a cluster of CTAs, each with its share of the channels (units of 16).
// One warp per source loads its units once, decodes them into shared memory (code *
// s_b, exact in f16) and takes the partial dots with every query; lane r of the warp
// puts them into CTA r's table (distributed shared memory), and one cluster barrier
// later every CTA sums the tables, forms the weights and mixes its own channels from
// the decoded rows.  One round trip to memory, one to the cluster (and before it a wait until
// every CTA runs, which the first source's loads cover).  One token, 4
// queries, 8 FP4 sources, d = 4096: 15.1 us in the streaming kernel (one CTA), 4.7 here.
#include "depth_cache.cuh"
#include "dispatch.h"

namespace attnres {

__device__ __forceinline__ uint32_t cf_map(const void *p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}

template <typename Tout, int FMT, int NQ>
__global__ void __launch_bounds__(CACHE_FEW_THREADS) cache_read_few_kernel(const CacheReadFewArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n_src = a.r.n_src, d = a.r.row.d, H = a.r.row.H, U = a.units, cs = a.cs;
    uint32_t *x = reinterpret_cast<uint32_t *>(smem);                       // [n_src][U * 8] f16x2
    float *part = reinterpret_cast<float *>(x + (size_t)n_src * U * 8);     // [cs][NQ][n_src], written by the cluster
    float *wt = part + cs * NQ * n_src;                                     // [NQ][n_src]
    float *tails = wt + NQ * n_src;                                         // [n_src][2]: row scale, sum of squares
    uint32_t rank;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    cluster_arrive_started();
    bool started = false;
    const int64_t t = blockIdx.x / cs;
    const int u0 = (int)rank * U, uph = d / 16 / H, head = u0 / uph;
    const unsigned char *tok = a.r.cache + t * a.r.row.bytes;

    for (int i = warp; i < n_src; i += CACHE_FEW_THREADS / 32) {
        const unsigned char *row = tok + (int64_t)i * a.r.cache_stride_bytes;
        if (lane < 2) tails[2 * i + lane] = __ldg(reinterpret_cast<const float *>(row + a.r.row.tail_off) + (lane ? 1 + head : 0));
        float2 dot[NQ];
#pragma unroll
        for (int q = 0; q < NQ; ++q) dot[q] = make_float2(0.f, 0.f);
        for (int u = lane; u < U; u += 32) {
            uint32_t xh[8];
            cache_unit_h2<FMT>(row, a.r.row, u0 + u, xh);
            uint4 *xs = reinterpret_cast<uint4 *>(x + ((size_t)i * U + u) * 8);
            xs[0] = make_uint4(xh[0], xh[1], xh[2], xh[3]);
            xs[1] = make_uint4(xh[4], xh[5], xh[6], xh[7]);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int c = (u0 + u) * 16 + 4 * v;
                float2 x0 = h2_to_f2(xh[2 * v]), x1 = h2_to_f2(xh[2 * v + 1]);
                if (a.r.gain) {
                    const float4 g = __ldg(reinterpret_cast<const float4 *>(a.r.gain + c));
                    x0 = fmul2(x0, make_float2(g.x, g.y));
                    x1 = fmul2(x1, make_float2(g.z, g.w));
                }
#pragma unroll
                for (int q = 0; q < NQ; ++q)
                    if (q < a.r.n_q) {
                        const float4 w = __ldg(reinterpret_cast<const float4 *>(a.r.queries + (size_t)q * d + c));
                        dot[q] = ffma2(x0, make_float2(w.x, w.y), dot[q]);
                        dot[q] = ffma2(x1, make_float2(w.z, w.w), dot[q]);
                    }
            }
        }
        if (!started) cluster_wait_started();
        started = true;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const float s = seg_sum<32>(dot[q].x + dot[q].y);
            if (lane < cs)
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cf_map(part + (rank * NQ + q) * n_src + i, lane)), "f"(s)
                             : "memory");
        }
    }
    if (!started) cluster_wait_started();      // (a warp without a source)
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");

    // weights: one warp per query; the partial dots of the CTAs that share this CTA's head
    const int r0 = head * uph / U, r1 = (head + 1) * uph / U;
    for (int q = warp; q < a.r.n_q; q += CACHE_FEW_THREADS / 32) {
        float m = -INFINITY;
        for (int i = lane; i < n_src; i += 32) {
            float s = 0.f;
            for (int r = r0; r < r1; ++r) s += part[(r * NQ + q) * n_src + i];
            s = cache_key_score(s, tails[2 * i + 1], 1.f / (float)(d / H), a.r.eps, tails[2 * i]);
            wt[q * n_src + i] = s;
            m = fmaxf(m, s);
        }
        m = seg_max<32>(m);
        float l = 0.f;
        for (int i = lane; i < n_src; i += 32) {
            const float e = __expf(wt[q * n_src + i] - m);
            l += e;
            wt[q * n_src + i] = e * tails[2 * i];
        }
        l = seg_sum<32>(l);
        const float inv = 1.f / l;
        for (int i = lane; i < n_src; i += 32) wt[q * n_src + i] *= inv;
        if (lane == 0 && (int)rank == r0 && a.r.lse) a.r.lse[((int64_t)q * H + head) * a.r.T + t] = m + __logf(l);
    }
    __syncthreads();
    for (int p = tid; p < U * 8; p += CACHE_FEW_THREADS) {
        float2 acc[NQ];
#pragma unroll
        for (int q = 0; q < NQ; ++q) acc[q] = make_float2(0.f, 0.f);
        for (int i = 0; i < n_src; ++i) {
            const float2 v = h2_to_f2(x[(size_t)i * U * 8 + p]);
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                if (q < a.r.n_q) {
                    const float w = wt[q * n_src + i];
                    acc[q] = ffma2(v, make_float2(w, w), acc[q]);
                }
        }
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            if (q < a.r.n_q) {
                unsigned char *o = a.r.out + q * a.r.out_q_stride_bytes + (t * d + u0 * 16 + 2 * p) * Elem<Tout>::BYTES;
                if constexpr (Elem<Tout>::BYTES == 2) *reinterpret_cast<uint32_t *>(o) = f2_to_bf2(acc[q].x, acc[q].y);
                else *reinterpret_cast<float2 *>(o) = acc[q];
            }
    }
}

template <typename T, int FMT>
static bool few_lookup(int nq, KernelRef *out) {
    switch (nq) {
        case 1: out->fn = reinterpret_cast<const void *>(&cache_read_few_kernel<T, FMT, 1>); return true;
        case 2: out->fn = reinterpret_cast<const void *>(&cache_read_few_kernel<T, FMT, 2>); return true;
        case 4: out->fn = reinterpret_cast<const void *>(&cache_read_few_kernel<T, FMT, 4>); return true;
        case 8: out->fn = reinterpret_cast<const void *>(&cache_read_few_kernel<T, FMT, 8>); return true;
    }
    return false;
}

bool lookup_cache_read_few(int dt, int fmt, int nq, KernelRef *out) {
    if (dt == 1) return fmt == CACHE_FP4 ? few_lookup<__nv_bfloat16, CACHE_FP4>(nq, out)
                                         : few_lookup<__nv_bfloat16, CACHE_FP8>(nq, out);
    return fmt == CACHE_FP4 ? few_lookup<float, CACHE_FP4>(nq, out) : few_lookup<float, CACHE_FP8>(nq, out);
}

}  // namespace attnres
