// Logits before a draw: repetition, presence and frequency penalties over a row's history, a bias,
// a grammar's bit mask, the temperature, and the log-softmax that the sampler reads, in one pass.
//
//   z = x + lse                         (x a log-probability row; without lse, x itself)
//   z = z > 0 ? z / rep : z * rep       for tokens of the history
//   z = z - presence [c > 0] - frequency c,  c the occurrences at and behind gen_start
//   z = z + bias;  z = -inf where the mask's bit is 0;  z = z / tau
//   out = z - log sum exp z
//
// Eight bytes per element (and four with a bias of every row) have to move; memory bounds it.  A
// row is cut over a cluster of CTAs, each of which keeps its share in registers between the two
// halves of the softmax, so the row is read once; every warp's (maximum, sum) goes to all CTAs of the
// cluster by distributed shared memory, and one cluster barrier per row joins them.  The clusters walk
// through the rows, and a thread's elements of the next row are on their way (cp.async, into places
// that only it reads) while this one's are reduced and written; a CTA per share without that spent
// most of its time waiting for its own loads (512 rows of 32768 with everything: 76 us).
// The history is counted into shared memory with integer atomics, whose order cannot change a
// count: bit 31 is set for a token seen anywhere, the bits below count the later part.
#include "paged.cuh"
#include "sm100.cuh"

namespace rlt {

namespace {

constexpr int MAX_CLUSTER = 8;
constexpr uint32_t SEEN = 0x80000000u;

constexpr float LOG2E = 1.4426950408889634f;
// 2^x by the ex2.approx instruction (relative error ~2^-22), a term of a sum only
__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <int BYTES>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}
template <int W>
__device__ __forceinline__ void load_w(const float* p, float* x) {
    if (W == 4) {
        const float4 q = *reinterpret_cast<const float4*>(p);
        x[0] = q.x; x[W > 1 ? 1 : 0] = q.y; x[W > 2 ? 2 : 0] = q.z; x[W > 2 ? 3 : 0] = q.w;
    } else {
        x[0] = *p;
    }
}

// LT threads with EPT elements each, in vectors of 4 (VEC) or one by one.  AHEAD: the next row's
// elements are fetched into shared memory (where that has room; one by one, each has a mask word too).
template <int LT, int EPT, bool VEC>
struct LogitsShape {
    static constexpr int W = VEC ? 4 : 1;
    static constexpr bool AHEAD = LT * EPT <= (VEC ? 16384 : 8192);
    static constexpr int CTAS = LT == 256 ? 4 : (LT * EPT <= 8192 ? 2 : 1);
    // counters; x, bias, mask words (one per vector) and a token per thread of the next row
    static size_t smem(int slice, bool history, bool bias) {
        return (size_t)slice * 4 * ((history ? 1 : 0) + (AHEAD ? 1 : 0) + (bias && AHEAD ? 1 : 0)) +
               (AHEAD ? (size_t)LT * (EPT / W + 1) * 4 : 0);
    }
};

template <int LT, int EPT, bool VEC>
__global__ void __launch_bounds__(LT, LogitsShape<LT, EPT, VEC>::CTAS) k_process_logits(LogitsArgs a, int slice, int n_cta) {
    using S = LogitsShape<LT, EPT, VEC>;
    constexpr int W = S::W, LW = LT / 32;
    extern __shared__ __align__(16) uint32_t count[];           // [slice] with a history
    float* ahead = reinterpret_cast<float*>(count + (a.tokens ? slice : 0));        // [slice] x of the next row
    float* bias_sm = ahead + slice;                             // [slice] its bias, or every row's
    uint32_t* mask_sm = reinterpret_cast<uint32_t*>(bias_sm + (a.bias ? slice : 0));    // [EPT / W][LT] its mask words
    int32_t* token_sm = reinterpret_cast<int32_t*>(mask_sm + EPT / W * LT);             // [LT] its first tokens
    __shared__ float2 pairs[2][MAX_CLUSTER * LW];               // of all warps of the cluster, by the row's parity
    const int rank = n_cta > 1 ? (int)cluster_rank() : 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int v0 = rank * slice, n = max(0, min(slice, a.V - v0));
    const int clusters = gridDim.x / n_cta;
    if (a.tokens)
        for (int i = tid; i < slice; i += LT) count[i] = 0;
    // a peer's shared memory may be written once the peer runs: the wait is before the first exchange
    if (n_cta > 1) cluster_arrive_release();
    pdl_wait();
    pdl_trigger();

    const bool own_bias = a.bias && a.bias_stride != 0;         // a bias of every row
    auto fetch = [&](long long b, bool bias_too) {
#pragma unroll
        for (int i = 0; i < EPT; i += W) {
            const int e = i * LT + tid * W;
            if (e >= n) continue;
            cp_async<4 * W>(ahead + e, a.x + b * a.x_stride + v0 + e);
            if (bias_too) cp_async<4 * W>(bias_sm + e, a.bias + b * a.bias_stride + v0 + e);
            if (a.mask) cp_async<4>(mask_sm + i / W * LT + tid, a.mask + b * a.mask_stride + ((v0 + e) >> 5));
        }
        if (a.tokens && tid < a.n_tokens) cp_async<4>(token_sm + tid, a.tokens + b * a.seq_stride + tid * a.tok_stride);
    };
    int b = blockIdx.x / n_cta;
    if (S::AHEAD) fetch(b, a.bias != nullptr);
    if (n_cta > 1) cluster_wait_acquire();
    else __syncthreads();                                       // the counters are zero

    for (int round = 0; b < a.B; b += clusters, ++round) {
        float rep = a.repetition ? a.repetition[b] : 1.f, tau = a.tau ? a.tau[b] : 1.f;
        const float presence = a.presence ? a.presence[b] : 0.f, frequency = a.frequency ? a.frequency[b] : 0.f;
        const float lse_in = a.lse ? a.lse[b] : 0.f;
        bool bad = false;
        if (!(rep > 0.f)) { rep = 1.f; bad = true; }
        if (!(tau > 0.f)) { tau = 1.f; bad = true; }
        if (S::AHEAD) cp_async_wait();                          // this thread's own elements
        if (a.tokens) {
            int len = a.tok_len ? a.tok_len[b] : a.n_tokens;
            if (len < 0 || len > a.n_tokens) { len = min(max(len, 0), a.n_tokens); bad = true; }
            const int gen = a.gen_start ? a.gen_start[b] : 0;
            const int32_t* t = a.tokens + b * a.seq_stride;
#pragma unroll 4
            for (int i = tid; i < len; i += LT) {
                const int id = S::AHEAD && i == tid ? token_sm[tid] : t[i * a.tok_stride], e = id - v0;
                if (id < 0 || id >= a.V) bad = true;
                else if (e >= 0 && e < n) {
                    if (i >= gen) atomicAdd(&count[e], 1u);
                    atomicOr(&count[e], SEEN);
                }
            }
            __syncthreads();
        }
        if (bad) raise_flag(a.hdr, ERR_BAD_LOGITS);

        const float inv_tau = 1.0f / tau, inv_rep = 1.0f / rep;
        float x[EPT];
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPT; i += W) {
            const int e = i * LT + tid * W;
#pragma unroll
            for (int j = 0; j < W; ++j) x[i + j] = 0.f;
            // the W elements of a vector lie in one word of the mask: their first id is a multiple of W
            uint32_t bits = e < n ? 0xfu : 0u;
            if (e < n) {
                if (a.mask) bits = (S::AHEAD ? mask_sm[i / W * LT + tid] : a.mask[b * a.mask_stride + ((v0 + e) >> 5)]) >> ((v0 + e) & 31);
                load_w<W>(S::AHEAD ? ahead + e : a.x + b * a.x_stride + v0 + e, x + i);
#pragma unroll
                for (int j = 0; j < W; ++j) x[i + j] += lse_in;
                if (a.tokens) {
                    uint32_t c[W], any = 0;
                    load_w<W>(reinterpret_cast<const float*>(count) + e, reinterpret_cast<float*>(c));
#pragma unroll
                    for (int j = 0; j < W; ++j) any |= c[j];
                    if (any) {
#pragma unroll
                        for (int j = 0; j < W; ++j) {
                            if (c[j]) {
                                x[i + j] *= x[i + j] > 0.f ? inv_rep : rep;
                                if (c[j] != SEEN) x[i + j] -= presence + frequency * (float)(c[j] & ~SEEN);
                                count[e + j] = 0;               // for the next row
                            }
                        }
                    }
                }
                if (a.bias) {
                    float bi[W];
                    load_w<W>(S::AHEAD ? bias_sm + e : a.bias + b * a.bias_stride + v0 + e, bi);
#pragma unroll
                    for (int j = 0; j < W; ++j) x[i + j] += bi[j];
                }
            }
#pragma unroll
            for (int j = 0; j < W; ++j) {
                x[i + j] = bits & (1u << j) ? x[i + j] * inv_tau : -INFINITY;
                m = fmaxf(m, x[i + j]);
            }
        }
        if (S::AHEAD && b + clusters < a.B) fetch(b + clusters, own_bias);

        m = warp_max(m);
        const float safe = m == -INFINITY ? 0.f : m;            // nothing allowed here: every term is exp(-inf)
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < EPT; ++i) s += ex2_approx((x[i] - safe) * LOG2E);       // (safe * LOG2E may overflow)
        s = warp_sum(s);
        float2* all = pairs[round & 1];
        if (n_cta > 1) {
            if (lane < n_cta) {
                const uint32_t to = cluster_addr(&all[rank * LW + warp], lane);
                asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(m), "f"(s) : "memory");
            }
            cluster_arrive_release();
            cluster_wait_acquire();
        } else {
            if (lane == 0) all[warp] = make_float2(m, s);
            __syncthreads();
        }
        // every warp joins the pairs alike
        m = -INFINITY;
        float2 mine[(MAX_CLUSTER * LW + 31) / 32];
#pragma unroll
        for (int k = 0; k < (MAX_CLUSTER * LW + 31) / 32; ++k) {
            const int i = k * 32 + lane;
            mine[k] = i < n_cta * LW ? all[i] : make_float2(-INFINITY, 0.f);
            m = fmaxf(m, mine[k].x);
        }
        m = warp_max(m);
        const float top = m == -INFINITY ? 0.f : m;
        s = 0.f;
#pragma unroll
        for (int k = 0; k < (MAX_CLUSTER * LW + 31) / 32; ++k) s += mine[k].y * ex2_approx((mine[k].x - top) * LOG2E);
        s = warp_sum(s);
        // No token allowed: all -inf.  (A NaN leaves no sum of zero, and the row is NaN.)
        const bool empty = m == -INFINITY && s == 0.f;
        const float log_s = empty ? 0.f : logf(s);
        if (rank == 0 && tid == 0) {
            if (a.out_lse) a.out_lse[b] = m + log_s;
            if (empty) raise_flag(a.hdr, ERR_BAD_LOGITS);
        }
        if (empty) m = 0.f;                                     // (its elements are -inf as they are)
        float* o = a.out + b * a.out_stride + v0;
#pragma unroll
        for (int i = 0; i < EPT; i += W) {
            const int e = i * LT + tid * W;
            if (e >= n) continue;
            float y[W];
#pragma unroll
            for (int j = 0; j < W; ++j) y[j] = x[i + j] - m - log_s;      // (m + log_s may round log_s away)
            if (VEC)
                __stcs(reinterpret_cast<float4*>(o + e), make_float4(y[0], y[W > 1 ? 1 : 0], y[W > 2 ? 2 : 0], y[W > 2 ? 3 : 0]));
            else
                o[e] = y[0];
        }
    }
}

template <int LT, int EPT, bool VEC>
cudaError_t run(Launch L, const LogitsArgs& a, int n_cta, int slice) {
    using S = LogitsShape<LT, EPT, VEC>;
    const size_t smem = S::smem(slice, a.tokens, a.bias);
    if (smem > 40 * 1024) {             // (the static part counts too)
        cudaError_t e = cudaFuncSetAttribute(k_process_logits<LT, EPT, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)S::smem(EPT * LT, true, true));
        if (e != cudaSuccess) return e;
    }
    // as many clusters as fit on the GPU at once, which then walk through the rows
    const int most = sm_count() * S::CTAS / n_cta, clusters = a.B < most ? a.B : most;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * n_cta));
    cfg.blockDim = dim3(LT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = L.pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)n_cta;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    *L.count += 1;
    return cudaLaunchKernelEx(&cfg, k_process_logits<LT, EPT, VEC>, a, slice, n_cta);
}

}  // namespace

int logits_max_vocab() { return MAX_CLUSTER * 64 * 512; }

cudaError_t launch_process_logits(Launch L, const LogitsArgs& a) {
    const auto al = [](const void* p, long long stride) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 4 == 0;
    };
    const bool vec = a.V % 4 == 0 && al(a.x, a.x_stride) && al(a.out, a.out_stride) &&
                     (!a.bias || al(a.bias, a.bias_stride));
    const auto share = [&](int c) { return ((a.V + c - 1) / c + 31) / 32 * 32; };
    // Every CTA more in a row's cluster costs time at its barrier (512 rows of 32768 with everything: 8
    // CTAs of 256 threads 70 us, 4 of 512 the same, 2 of 1024 50 us), so rows are cut as little as
    // possible where there are enough of them for every SM ...
    const int c1 = (a.V + 16383) / 16384;
    if (a.V > 2048 && a.V <= 8192 && a.B >= 2 * sm_count())
        return vec ? run<512, 16, true>(L, a, 1, share(1)) : run<512, 16, false>(L, a, 1, share(1));
    if (a.V > 2048 && c1 <= MAX_CLUSTER && (long long)a.B * c1 >= sm_count())
        return vec ? run<1024, 16, true>(L, a, c1, share(c1)) : run<1024, 16, false>(L, a, c1, share(c1));
    // ... and else until there are two CTAs of 256 threads per SM, while every thread keeps 8 elements
    // (64 rows of 32000: 9 us against 13 us).
    int c = (a.V + 4095) / 4096;
    if (c <= MAX_CLUSTER) {
        while (c < MAX_CLUSTER && a.B * c < 2 * sm_count() && a.V >= c * 2048) ++c;
        const int ept = (share(c) + 255) / 256;
        if (ept <= 4) return vec ? run<256, 4, true>(L, a, c, share(c)) : run<256, 4, false>(L, a, c, share(c));
        if (ept <= 8) return vec ? run<256, 8, true>(L, a, c, share(c)) : run<256, 8, false>(L, a, c, share(c));
        return vec ? run<256, 16, true>(L, a, c, share(c)) : run<256, 16, false>(L, a, c, share(c));
    }
    // few rows of large vocabularies
    const int ept = (share(MAX_CLUSTER) + 511) / 512;
    c = MAX_CLUSTER;
    if (ept <= 16) return vec ? run<512, 16, true>(L, a, c, share(c)) : run<512, 16, false>(L, a, c, share(c));
    return vec ? run<512, 64, true>(L, a, c, share(c)) : run<512, 64, false>(L, a, c, share(c));
}

}  // namespace rlt
