// Logits before a draw: repetition, presence and frequency penalties over a row's history, a bias,
// a grammar's bit mask, the temperature, and the log-softmax that the sampler reads, in one pass.
//
//   z = x + lse                         (x a log-probability row; without lse, x itself)
//   z = z > 0 ? z / rep : z * rep       for tokens of the history
//   z = z - presence [c > 0] - frequency c,  c the occurrences at and behind gen_start
//   z = z + bias;  z = -inf where the mask's bit is 0;  z = z / tau
//   out = z - log sum exp z
//
// Eight bytes per element (and four with a bias of every row) have to move; memory bounds it where rows
// are many, and the chain of steps per row where they are few.  A row is cut over a cluster of CTAs,
// each of which keeps its share in registers between the two halves of the softmax, so the row is read
// once; every warp's (maximum, sum) goes to all CTAs of the cluster by distributed shared memory, and one
// cluster barrier per row joins them.  The clusters walk through the rows, and a thread's elements of the
// next row are on their way (cp.async) while this one's are reduced and written.  Two CTAs per SM work
// while the other waits, and few threads with many elements each spend less on what a row costs a warp:
// 512 rows of 32768 with everything take 42 us by pairs of 256 threads with 64 elements each, 44 by 1024
// with 16, one CTA per SM, and 76 without the copies ahead.
//
// Divisions by the temperature and the repetition are products with their reciprocals, and the sum's
// exponentials are ex2.approx (2^-22 each): beside the formula's own float32 roundings both are small (error
// against 64 bits 5e-8 of the norm in place of 4.4e-8 for one row of 512, 3.7e-8 and 3.9e-8 for 512 of 32768).
//
// The history is counted into shared memory with integer atomics, whose order cannot change a count.
// Of a token's occurrences the one that comes first then changes its logit, so that the steps over the
// whole row know nothing of penalties (looking at every element's counter took 47 us in place of 44).
#include <cfloat>

#include "paged.cuh"
#include "sm100.cuh"

namespace rlt {

namespace {

constexpr int MAX_CLUSTER = 8;
constexpr uint32_t SEEN = 0x80000000u;      // in a counter of 32 bits
constexpr uint32_t DONE = 0xffffu;          // in one of 16 bits, which counts up to MAX_COUNT
constexpr int MAX_COUNT = 0xfffe;
constexpr int TOKENS = 1024;                // of a history, fetched ahead

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
// elements are fetched into shared memory (where that has room), and counters have 16 bits.
template <int LT, int EPT, bool VEC>
struct LogitsShape {
    static constexpr int W = VEC ? 4 : 1;
    static constexpr bool AHEAD = LT * EPT <= 16384;
    static constexpr bool BIAS = LT * EPT <= 8192;              // the bias too
    static constexpr int CTAS = LT * EPT <= 4096 ? 4 : (LT * EPT <= 16384 ? 2 : 1);
    static constexpr int WORDS = LT * EPT / 32;                 // of the mask
    // counters; x, bias, mask words (of two rows) and the first tokens of the next row
    static size_t smem(int slice, bool history, bool bias) {
        return (size_t)slice * ((history ? (AHEAD ? 2 : 4) : 0) + (AHEAD ? 4 : 0) + (bias && BIAS ? 4 : 0)) +
               (AHEAD ? (size_t)(2 * WORDS + TOKENS) * 4 : 0);
    }
};

// What a call asks of a row.
struct LogitsRow {
    float rep, tau, presence, frequency, lse;
    int len, gen;
};
__device__ __forceinline__ LogitsRow load_row(const LogitsArgs& a, int b) {
    return {a.repetition ? a.repetition[b] : 1.f, a.tau ? a.tau[b] : 1.f, a.presence ? a.presence[b] : 0.f,
            a.frequency ? a.frequency[b] : 0.f, a.lse ? a.lse[b] : 0.f, a.tok_len ? a.tok_len[b] : a.n_tokens,
            a.gen_start ? a.gen_start[b] : 0};
}

// A repetition or a temperature: a normal number above 0, so that its reciprocal is finite.
__device__ __forceinline__ bool factor_ok(float x) { return x >= FLT_MIN && x <= FLT_MAX; }

template <int LT, int EPT, bool VEC>
__global__ void __launch_bounds__(LT, LogitsShape<LT, EPT, VEC>::CTAS) k_process_logits(LogitsArgs a, int slice, int n_cta) {
    using S = LogitsShape<LT, EPT, VEC>;
    constexpr int W = S::W, LW = LT / 32;
    extern __shared__ __align__(16) uint32_t count[];           // [slice] with a history
    uint16_t* const count16 = reinterpret_cast<uint16_t*>(count);
    float* ahead = reinterpret_cast<float*>(count + (a.tokens ? slice / 2 : 0));    // [slice] x of the next row
    float* bias_sm = ahead + slice;                             // [slice] its bias, or every row's
    // [2][WORDS] mask words, by the row's parity
    uint32_t* mask_sm = reinterpret_cast<uint32_t*>(bias_sm + (S::BIAS && a.bias ? slice : 0));
    int32_t* token_sm = reinterpret_cast<int32_t*>(mask_sm + 2 * S::WORDS);             // [TOKENS] its first tokens
    __shared__ float2 pairs[2][MAX_CLUSTER * LW];               // of all warps of the cluster, by the row's parity
    const int rank = n_cta > 1 ? (int)cluster_rank() : 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int v0 = rank * slice, n = max(0, min(slice, a.V - v0));
    const int clusters = gridDim.x / n_cta;
    if (a.tokens)
        for (int i = tid; i < (S::AHEAD ? slice / 2 : slice); i += LT) count[i] = 0;
    // a peer's shared memory may be written once the peer runs: the wait is before the first exchange
    if (n_cta > 1) cluster_arrive_release();
    pdl_wait();
    pdl_trigger();

    const bool own_bias = a.bias && a.bias_stride != 0;         // a bias of every row
    auto fetch = [&](long long b, int parity, bool bias_too) {
        const float* x = a.x + b * a.x_stride + v0 + tid * W;
        const float* bias = a.bias + b * a.bias_stride + v0 + tid * W;
#pragma unroll
        for (int i = 0; i < EPT; i += W) {
            if (i * LT + tid * W >= n) continue;
            cp_async<4 * W>(ahead + tid * W + i * LT, x + i * LT);
            if (S::BIAS && bias_too) cp_async<4 * W>(bias_sm + tid * W + i * LT, bias + i * LT);
        }
        if (a.mask)
            for (int i = tid; i * 32 < n; i += LT)
                cp_async<4>(mask_sm + parity * S::WORDS + i, a.mask + b * a.mask_stride + (v0 >> 5) + i);
        if (a.tokens)
            for (int i = tid; i < min(a.n_tokens, TOKENS); i += LT)
                cp_async<4>(token_sm + i, a.tokens + b * a.seq_stride + i * a.tok_stride);
    };
    int b = blockIdx.x / n_cta;
    if (S::AHEAD) fetch(b, 0, a.bias != nullptr);
    LogitsRow row = load_row(a, b);
    if (n_cta > 1) cluster_wait_acquire();
    else __syncthreads();                                       // the counters are zero

    for (int round = 0; b < a.B; b += clusters, ++round) {
        bool bad = false;
        if (!factor_ok(row.rep)) { row.rep = 1.f; bad = true; }
        if (!factor_ok(row.tau)) { row.tau = 1.f; bad = true; }
        if (row.len < 0 || row.len > a.n_tokens) { row.len = min(max(row.len, 0), a.n_tokens); bad = true; }
        const float inv_tau = 1.0f / row.tau, inv_rep = 1.0f / row.rep, lse_in = row.lse;
        const float to_log2 = inv_tau * LOG2E;                  // (inv_tau is 2^126 at most)
        // Less the input's log-sum-exp, as x is: only penalties need it, the softmax does not.
        auto penalise = [&](float x, uint32_t c) {
            x += lse_in;
            const float y = x * (x > 0.f ? inv_rep : row.rep);
            // what the penalty takes out of float32's range stays at its end
            x = isinf(y) && !isinf(x) ? copysignf(FLT_MAX, x) : y;
            if (c > 0) x -= row.presence + row.frequency * (float)c;
            return x - lse_in;
        };
        const int32_t* t = a.tokens + b * a.seq_stride;
        auto each_token = [&](auto&& visit) {                   // of the history, in this CTA's share
#pragma unroll 2
            for (int i = tid; i < row.len; i += LT) {
                const int id = S::AHEAD && i < TOKENS ? token_sm[i] : t[i * a.tok_stride], e = id - v0;
                if (id < 0 || id >= a.V) bad = true;
                else if (e >= 0 && e < n) visit(i, e);
            }
        };
        if (S::AHEAD) cp_async_wait();
        if (a.tokens) {
            each_token([&](int i, int e) {
                if (S::AHEAD) {
                    if (i >= row.gen) atomicAdd(&count[e >> 1], 1u << 16 * (e & 1));
                } else {
                    if (i >= row.gen) atomicAdd(&count[e], 1u);
                    atomicOr(&count[e], SEEN);
                }
            });
            __syncthreads();
            if (S::AHEAD) {
                // whoever of a token's occurrences comes first sees to it
                each_token([&](int, int e) {
                    const uint32_t c = atomicOr(&count[e >> 1], DONE << 16 * (e & 1)) >> 16 * (e & 1) & DONE;
                    if (c != DONE) ahead[e] = penalise(ahead[e], c);
                });
                __syncthreads();
                each_token([&](int, int e) { count16[e] = 0; });        // for the next row
            }
        } else if (S::AHEAD && a.mask) {
            __syncthreads();
        }
        if (bad) raise_flag(a.hdr, ERR_BAD_LOGITS);

        // Steps without a branch per element: what lies behind the share is read too, from somewhere in
        // it, and made -inf at the end.
        float x[EPT];
#pragma unroll
        for (int i = 0; i < EPT; i += W) {
            const int e = i * LT + tid * W;
            if (S::AHEAD) {
                load_w<W>(ahead + min(e, slice - W), x + i);
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) x[i + j] = 0.f;
                if (e < n) load_w<W>(a.x + b * a.x_stride + v0 + e, x + i);
                if (e < n && a.tokens) {
                    uint32_t c[W], any = 0;
                    load_w<W>(reinterpret_cast<const float*>(count) + e, reinterpret_cast<float*>(c));
#pragma unroll
                    for (int j = 0; j < W; ++j) any |= c[j];
                    if (any) {
#pragma unroll
                        for (int j = 0; j < W; ++j) {
                            if (c[j]) {
                                x[i + j] = penalise(x[i + j], c[j] & ~SEEN);
                                count[e + j] = 0;               // for the next row
                            }
                        }
                    }
                }
            }
        }
        if (a.bias) {
#pragma unroll
            for (int i = 0; i < EPT; i += W) {
                const int e = i * LT + tid * W;
                float bi[W];
#pragma unroll
                for (int j = 0; j < W; ++j) bi[j] = 0.f;
                if (S::BIAS) load_w<W>(bias_sm + min(e, slice - W), bi);
                else if (e < n) load_w<W>(a.bias + b * a.bias_stride + v0 + e, bi);
#pragma unroll
                for (int j = 0; j < W; ++j) x[i + j] += bi[j];
            }
        }
        if (a.mask) {
#pragma unroll
            for (int i = 0; i < EPT; i += W) {
                // the W elements of a vector lie in one word: their first id is a multiple of W
                const int e = i * LT + tid * W;
                uint32_t word = 0;
                if (S::AHEAD) word = mask_sm[(round & 1) * S::WORDS + (e >> 5)];
                else if (e < n) word = a.mask[b * a.mask_stride + ((v0 + e) >> 5)];
                word >>= tid * W & 31;
#pragma unroll
                for (int j = 0; j < W; ++j) x[i + j] = word & (1u << j) ? x[i + j] : -INFINITY;
            }
        }
        if (n < LT * EPT) {
#pragma unroll
            for (int i = 0; i < EPT; i += W)
#pragma unroll
                for (int j = 0; j < W; ++j) x[i + j] = i * LT + tid * W < n ? x[i + j] : -INFINITY;
        }
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPT; ++i) m = fmaxf(m, x[i]);
        if (b + clusters < a.B) {
            if (S::AHEAD) fetch(b + clusters, (round + 1) & 1, own_bias);
            row = load_row(a, b + clusters);
        }

        m = warp_max(m);
        const float safe = m == -INFINITY ? 0.f : m;            // nothing allowed here: every term is exp(-inf)
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < EPT; i += 2) {
            // the maximum is taken off before the scale: neither x / tau nor safe / tau need be in range
            const float2 y = mul2(add2(make_float2(x[i], x[i + 1]), make_float2(-safe, -safe)), make_float2(to_log2, to_log2));
            sum = add2(sum, make_float2(ex2_approx(y.x), ex2_approx(y.y)));
        }
        float s = warp_sum(sum.x + sum.y);
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
        for (int i = lane; i < n_cta * LW; i += 32) m = fmaxf(m, all[i].x);
        m = warp_max(m);
        const float top = m == -INFINITY ? 0.f : m;
        s = 0.f;
        for (int i = lane; i < n_cta * LW; i += 32) s += all[i].y * ex2_approx((all[i].x - top) * to_log2);
        s = warp_sum(s);
        // No token allowed: all -inf.  (A NaN leaves no sum of zero, and the row is NaN.)
        const bool empty = m == -INFINITY && s == 0.f;
        const float log_s = (empty ? 0.f : logf(s)) + (lse_in - lse_in);        // (NaN where lse is)
        if (rank == 0 && tid == 0) {
            if (a.out_lse) a.out_lse[b] = (m + lse_in) * inv_tau + log_s;
            if (empty) raise_flag(a.hdr, ERR_BAD_LOGITS);
        }
        if (empty) m = 0.f;                                     // (its elements are -inf as they are)
        float* o = a.out + b * a.out_stride + v0;
#pragma unroll
        for (int i = 0; i < EPT; i += W) {
            const int e = i * LT + tid * W;
            if (e >= n) continue;
            // (m / tau + log_s may round log_s away)
            if (VEC) {
                const float2 mm = make_float2(-m, -m), tt = make_float2(inv_tau, inv_tau), ll = make_float2(-log_s, -log_s);
                const float2 y0 = fma2(add2(make_float2(x[i], x[i + 1]), mm), tt, ll);
                const float2 y1 = fma2(add2(make_float2(x[i + W / 2], x[i + W - 1]), mm), tt, ll);
                __stcs(reinterpret_cast<float4*>(o + e), make_float4(y0.x, y0.y, y1.x, y1.y));
            } else {
                o[e] = fmaf(x[i] - m, inv_tau, -log_s);
            }
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
    // Counters of 16 bits could overflow.
    if (a.tokens && a.n_tokens > MAX_COUNT) {
        const int c = (a.V + 32767) / 32768;
        return vec ? run<512, 64, true>(L, a, c, share(c)) : run<512, 64, false>(L, a, c, share(c));
    }
    // Every CTA more in a row's cluster costs time at its barrier (512 rows of 32768 with everything: 4
    // CTAs of 256 threads 54 us, 2 of them 42 us), so rows are cut as little as possible where that gives
    // every second SM a CTA (64 rows of 32000: 2 CTAs 8.9 us, 8 of them 9.9 us; 16 rows: 8.5 us, 6.5 us) ...
    const auto enough = [&](int c) { return 2LL * a.B * c >= sm_count(); };
    const int c1 = (a.V + 16383) / 16384;
    // (100 rows of 8192: one CTA 6.1 us, three 8.3 us; rows up to 4096 have smaller ones below)
    if (a.V > 4096 && a.V <= 8192 && enough(1))
        return vec ? run<512, 16, true>(L, a, 1, share(1)) : run<512, 16, false>(L, a, 1, share(1));
    if (a.V > 8192 && c1 <= MAX_CLUSTER && enough(c1))
        return vec ? run<256, 64, true>(L, a, c1, share(c1)) : run<256, 64, false>(L, a, c1, share(c1));
    // ... and else until there are as many, while every thread keeps 8 elements
    int c = (a.V + 4095) / 4096;
    if (c <= MAX_CLUSTER) {
        while (c < MAX_CLUSTER && !enough(c) && a.V >= c * 2048) ++c;
        const int ept = (share(c) + 255) / 256;
        if (ept <= 4) return vec ? run<256, 4, true>(L, a, c, share(c)) : run<256, 4, false>(L, a, c, share(c));
        if (ept <= 8) return vec ? run<256, 8, true>(L, a, c, share(c)) : run<256, 8, false>(L, a, c, share(c));
        return vec ? run<256, 16, true>(L, a, c, share(c)) : run<256, 16, false>(L, a, c, share(c));
    }
    // few rows of large vocabularies (4 rows of 131072: 8.5 us, by 512 threads with 64 elements 11.7 us)
    c = MAX_CLUSTER;
    if (share(c) <= 512 * 16) return vec ? run<512, 16, true>(L, a, c, share(c)) : run<512, 16, false>(L, a, c, share(c));
    if (c1 <= c) return vec ? run<256, 64, true>(L, a, c, share(c)) : run<256, 64, false>(L, a, c, share(c));
    return vec ? run<512, 64, true>(L, a, c, share(c)) : run<512, 64, false>(L, a, c, share(c));
}

}  // namespace rlt
