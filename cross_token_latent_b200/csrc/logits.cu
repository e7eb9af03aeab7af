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
// halves of the softmax, so the row is read once; (maximum, sum) pairs cross by distributed shared
// memory.  The history is counted into shared memory with integer atomics, whose order cannot
// change a count: bit 31 is set for a token seen anywhere, the bits below count the later part.
#include <cooperative_groups.h>

#include "paged.cuh"
#include "sm100.cuh"

namespace rlt {

namespace {

namespace cg = cooperative_groups;

constexpr int LT = 512;                 // threads
constexpr int LW = LT / 32;
constexpr int MAX_CLUSTER = 8;
constexpr uint32_t SEEN = 0x80000000u;

// EPT elements per thread, in vectors of 4 (VEC) or one by one.
template <int EPT, bool VEC>
__global__ void __launch_bounds__(LT) k_process_logits(LogitsArgs a, int slice) {
    extern __shared__ uint32_t count[];             // [slice], with a history only
    __shared__ float red[2][LW];
    __shared__ float2 peers[MAX_CLUSTER];
    cg::cluster_group cluster = cg::this_cluster();
    const int n_cta = cluster.num_blocks(), rank = cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / n_cta;
    const int v0 = rank * slice, n = max(0, min(slice, a.V - v0));
    constexpr int W = VEC ? 4 : 1;
    if (a.tokens)
        for (int i = tid; i < n; i += LT) count[i] = 0;
    // a peer's shared memory may be written once the peer runs: the wait is before the exchange
    if (n_cta > 1) cluster_arrive_relaxed();
    pdl_wait();
    pdl_trigger();

    float x[EPT];
    const float* row = a.x + b * a.x_stride + v0;
#pragma unroll
    for (int i = 0; i < EPT; i += W) {
        const int e = i * LT + tid * W;
        if (VEC) {
            const float4 q = e < n ? __ldcs(reinterpret_cast<const float4*>(row + e)) : make_float4(0, 0, 0, 0);
            x[i] = q.x;
            if (W > 1) { x[i + 1] = q.y; x[i + 2] = q.z; x[i + 3] = q.w; }
        } else {
            x[i] = e < n ? __ldcs(row + e) : 0.f;
        }
    }
    float rep = a.repetition ? a.repetition[b] : 1.f, tau = a.tau ? a.tau[b] : 1.f;
    const float presence = a.presence ? a.presence[b] : 0.f, frequency = a.frequency ? a.frequency[b] : 0.f;
    const float lse_in = a.lse ? a.lse[b] : 0.f;
    bool bad = false;
    if (!(rep > 0.f)) { rep = 1.f; bad = true; }
    if (!(tau > 0.f)) { tau = 1.f; bad = true; }
    if (a.tokens) {
        int len = a.tok_len ? a.tok_len[b] : a.n_tokens;
        if (len < 0 || len > a.n_tokens) { len = min(max(len, 0), a.n_tokens); bad = true; }
        const int gen = a.gen_start ? a.gen_start[b] : 0;
        const int32_t* t = a.tokens + b * a.seq_stride;
        __syncthreads();                            // the counters are zero
        for (int i = tid; i < len; i += LT) {
            const int id = t[i * a.tok_stride];
            if (id < 0 || id >= a.V) { bad = true; continue; }
            const int e = id - v0;
            if (e < 0 || e >= n) continue;
            if (i >= gen) atomicAdd(&count[e], 1u);
            atomicOr(&count[e], SEEN);
        }
        __syncthreads();
    }
    if (bad) raise_flag(a.hdr, ERR_BAD_LOGITS);

    const float inv_tau = 1.0f / tau;
    const float* bias = a.bias ? a.bias + b * a.bias_stride + v0 : nullptr;
    const uint32_t* mask = a.mask ? a.mask + b * a.mask_stride : nullptr;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPT; i += W) {
        const int e = i * LT + tid * W;
        float bi[W];
        uint32_t bits = 0xfu;
        if (e < n) {
            if (bias) {
                if (VEC) {
                    const float4 q = *reinterpret_cast<const float4*>(bias + e);
                    bi[0] = q.x;
                    if (W > 1) { bi[W > 1 ? 1 : 0] = q.y; bi[W > 1 ? 2 : 0] = q.z; bi[W > 1 ? 3 : 0] = q.w; }
                } else {
                    bi[0] = bias[e];
                }
            }
            // the W elements lie in one word: their first id is a multiple of W
            if (mask) bits = mask[(v0 + e) >> 5] >> ((v0 + e) & 31);
        } else {
            bits = 0;
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float z = x[i + j] + lse_in;
            if (a.tokens && e < n) {
                const uint32_t c = count[e + j];
                if (c) {
                    const float k = (float)(c & ~SEEN);
                    z = z > 0.f ? z / rep : z * rep;
                    if (c != SEEN) z -= presence + frequency * k;
                }
            }
            if (bias && e < n) z += bi[j];
            z *= inv_tau;
            if (!((bits >> j) & 1u)) z = -INFINITY;
            x[i + j] = z;
            m = fmaxf(m, z);
        }
    }
    m = warp_max(m);
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
    m = warp_max(lane < LW ? red[0][lane] : -INFINITY);
    const float safe = m == -INFINITY ? 0.f : m;    // nothing allowed here: every term is exp(-inf)
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < EPT; ++i) s += expf(x[i] - safe);
    s = warp_sum(s);
    if (lane == 0) red[1][warp] = s;
    __syncthreads();
    s = warp_sum(lane < LW ? red[1][lane] : 0.f);
    if (n_cta > 1) {
        cluster_wait_acquire();
        if (tid < n_cta) *cluster.map_shared_rank(&peers[rank], tid) = make_float2(m, s);
        cluster.sync();
        float mt = -INFINITY;
        for (int j = 0; j < n_cta; ++j) mt = fmaxf(mt, peers[j].x);
        const float st = mt == -INFINITY ? 0.f : mt;
        s = 0.f;
        for (int j = 0; j < n_cta; ++j) s += peers[j].y * expf(peers[j].x - st);
        m = mt;
    }
    // No token allowed: all -inf.  (A NaN leaves no sum of zero, and the row is NaN.)
    const bool empty = m == -INFINITY && s == 0.f;
    const float lse = empty ? -INFINITY : m + logf(s);
    if (rank == 0 && tid == 0) {
        if (a.out_lse) a.out_lse[b] = lse;
        if (empty) raise_flag(a.hdr, ERR_BAD_LOGITS);
    }
    float* o = a.out + b * a.out_stride + v0;
#pragma unroll
    for (int i = 0; i < EPT; i += W) {
        const int e = i * LT + tid * W;
        if (e >= n) continue;
        float y[W];
#pragma unroll
        for (int j = 0; j < W; ++j) y[j] = empty ? -INFINITY : x[i + j] - lse;
        if (VEC)
            *reinterpret_cast<float4*>(o + e) = make_float4(y[0], y[W > 1 ? 1 : 0], y[W > 1 ? 2 : 0], y[W > 1 ? 3 : 0]);
        else
            o[e] = y[0];
    }
}

template <int EPT, bool VEC>
cudaError_t run(Launch L, const LogitsArgs& a, int clusters, int slice) {
    const size_t smem = a.tokens ? (size_t)slice * 4 : 0;
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(k_process_logits<EPT, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             EPT * LT * 4);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * clusters));
    cfg.blockDim = dim3(LT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = L.pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)clusters;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    *L.count += 1;
    return cudaLaunchKernelEx(&cfg, k_process_logits<EPT, VEC>, a, slice);
}

}  // namespace

int logits_max_vocab() { return MAX_CLUSTER * 64 * LT; }

cudaError_t launch_process_logits(Launch L, const LogitsArgs& a) {
    // A CTA's share is at most 16 elements per thread where eight CTAs can do that (registers for
    // two CTAs per SM and more), and rows are cut further while the grid is below two CTAs per SM
    // and a share keeps an element or two for every thread.
    int c = 1;
    while (c < MAX_CLUSTER && (a.V > c * 16 * LT || (a.B * c < 2 * sm_count() && a.V >= c * 4 * LT))) c *= 2;
    const int slice = ((a.V + c - 1) / c + 31) / 32 * 32;
    const int ept = (slice + LT - 1) / LT;
    const auto al = [](const void* p, long long stride) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 4 == 0;
    };
    const bool vec = a.V % 4 == 0 && al(a.x, a.x_stride) && al(a.out, a.out_stride) &&
                     (!a.bias || al(a.bias, a.bias_stride));
    if (ept <= 8) return vec ? run<8, true>(L, a, c, slice) : run<8, false>(L, a, c, slice);
    if (ept <= 16) return vec ? run<16, true>(L, a, c, slice) : run<16, false>(L, a, c, slice);
    if (ept <= 32) return vec ? run<32, true>(L, a, c, slice) : run<32, false>(L, a, c, slice);
    return vec ? run<64, true>(L, a, c, slice) : run<64, false>(L, a, c, slice);
}

}  // namespace rlt
