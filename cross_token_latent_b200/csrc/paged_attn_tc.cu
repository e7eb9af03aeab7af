// Attention of many new rows over a paged cache on the sm_100a tensor cores (bf16, head_dim 64 or
// 128).  A CTA (one per SM, two at head width 64) takes an equal share of all the work (paged.cuh) and
// walks through the items in it.  An item is a tile of one key head's rows, two stages of up to 128 (rows of a group of query
// heads beside each other, so that shared keys are read once), against key tiles of 128:
//   warps 0-3    softmax of stage 0, warps 4-7 of stage 1, a thread per row: the scores leave TMEM
//                once, P_s goes back as bf16 over the scores' own columns
//   warp 8       TMA producer: an item's query tiles, then K and V tiles alternately into a ring; a
//                tile is as many boxes as it has pages, one lane each
//   warp 9       the MMAs, stage 0 and 1 in turn: O_s += P_s V with P_s read from TMEM and V as it lies
//                in the page (MN-major), then the next S_s = Q_s K^T into the stage's 128 TMEM columns.
//                One elected thread issues, which keeps the descriptors in uniform registers (a thread
//                that the compiler does not know to be alone took some 95 clocks per MMA).  A warp per
//                stage was slower: their products interleave, both softmaxes fall in step and the
//                tensor core idles meanwhile
//   warp 10      clears the end of a last V tile
// While one stage's rows are in the softmax the tensor core works on the other stage, and an item's
// last products and its output overlap with the next one's first loads and scores.  The running
// maximum moves only when it grew by more than 2^8 (RESCALE): a smaller maximum is as good a
// reference for the exponentials, and the accumulator then seldom has to be rescaled; a stage's O is
// final when its next scores have arrived, because its MMAs complete in order.  (Rescaling seldom, and
// taking part of the exponentials on the multiply-add units, are published techniques of attention kernels
// for these tensor cores.)
// Probabilities are rounded to bf16 for the product, as the tensor core takes them (2^-8 each at most), and
// their sum is of the rounded values, so that the result stays a weighted mean of the values (a row of few
// keys was off by up to 2^-8 more with the sum of the unrounded ones, which took 716 us for the long chunk
// below).  O, maximum and sum are float32.
// What bounds it is the softmax: 8192 tokens of 16 heads of 128 behind 8192 others take 738 us, 1117
// TFLOP/s or 68 % of the tensor cores' measured rate (tensor pipe 59 % of the cycles, special function
// unit 45 %, issue 48 %: the chain of a stage, no single pipe); heads of 64 take 561 us for half the
// operations (35 %, 53 %, 63 %).
// Every mbarrier wait is bounded.
#include "paged.cuh"
#include "sm100.cuh"

namespace rlt {

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int KT = 128;                 // keys per tile of the ring
constexpr float RESCALE = 8.0f;         // log2: probabilities stay below 256

template <int HD>
struct TcShape {
    static constexpr int STAGES = PAGED_TC_STAGES;          // of up to 128 rows
    static constexpr int CTAS = paged_tc_ctas(HD);          // per SM
    static constexpr int KH = HD;                           // keys per block of scores
    static constexpr int NB = KT / KH;                      // blocks per key tile
    static constexpr int ATOMS = HD / 64;                   // 64-element swizzle atoms of a row
    static constexpr int Q_BYTES = 128 * HD * 2;            // one stage
    static constexpr int T_BYTES = KT * HD * 2;             // a tile of K or V
    static constexpr int SLOTS = HD == 128 ? 5 : 4;
    static constexpr int OFF_KV = STAGES * Q_BYTES;
    static constexpr int OFF_BAR = OFF_KV + SLOTS * T_BYTES;
    static constexpr int SMEM = OFF_BAR + 256 + 1024;
    static constexpr int POLY = 2;                          // of 8 exponentials, those not on the special function unit
    static constexpr uint32_t O_COL = STAGES * KH;          // O behind the scores
    static constexpr uint32_t TMEM_COLS = STAGES * (KH + HD);
    static constexpr int SOFTMAX_WARPS = 4 * STAGES;
    static constexpr int PRODUCER = SOFTMAX_WARPS, ISSUER = SOFTMAX_WARPS + 1, CLEARER = SOFTMAX_WARPS + 2;
    static constexpr int THREADS = (SOFTMAX_WARPS + 3) * 32;
};

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One thread of a converged warp, known as such to the compiler: the descriptors of the MMAs that it
// issues then stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

// 2^x for two x in [-125, 0] and a little above on the multiply-add units: x = n + f with n the nearest
// whole number, 2^f by the polynomial of degree 3 with the smallest relative error on [-1/2, 1/2]
// (equal ripple, 2^-13.7; the results are rounded to bf16), n added to the exponent.  The special
// function unit gives 16 exponentials a clock and would hold the tensor core up.
__device__ __forceinline__ float2 ex2_poly(float2 x) {
    x.x = fmaxf(x.x, -125.f);
    x.y = fmaxf(x.y, -125.f);
    const float big = 12582912.f;                   // 1.5 * 2^23: a sum's low bits are the whole part
    const float2 t = add2(x, make_float2(big, big));
    const float2 n = add2(t, make_float2(-big, -big));
    const float2 f = fma2(n, make_float2(-1.f, -1.f), x);
    float2 r = fma2(f, make_float2(0.05517166852951050f, 0.05517166852951050f),
                    make_float2(0.24261112511157990f, 0.24261112511157990f));
    r = fma2(r, f, make_float2(0.69326096773147583f, 0.69326096773147583f));
    r = fma2(r, f, make_float2(0.99992805719375610f, 0.99992805719375610f));
    r.x = __int_as_float(__float_as_int(r.x) + (__float_as_int(t.x) << 23));
    r.y = __int_as_float(__float_as_int(r.y) + (__float_as_int(t.y) << 23));
    return r;
}

// s += the two bf16 halves of w, in float32.  (Shifting and masking them into place: 746 us in place of 737
// for the long chunk, 570 in place of 560 with heads of 64.)
__device__ __forceinline__ void add_bf16x2(float2& s, uint32_t w) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "add.rn.f32.bf16 %0, l, %0;\n\tadd.rn.f32.bf16 %1, h, %1;\n\t}"
        : "+f"(s.x), "+f"(s.y)
        : "r"(w));
}

// Probabilities of 32 scores (of scaled scores less the maximum, bf16, two to a word) into the TMEM
// columns at t_p, and the sum of what was stored.  POLY of every 8 pairs take the polynomial.
template <int POLY>
__device__ __forceinline__ float softmax32(const uint32_t (&x)[32], uint32_t t_p, float c2, float neg) {
    const float2 cc = make_float2(c2, c2), nn = make_float2(neg, neg);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    uint32_t pk[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float2 y = fma2(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), cc, nn);
        if (i % 8 * POLY / 8 != (i % 8 + 1) * POLY / 8) {
            y = ex2_poly(y);
        } else {
            y.x = ex2_approx(y.x);
            y.y = ex2_approx(y.y);
        }
        __nv_bfloat162 h = __floats2bfloat162_rn(y.x, y.y);
        pk[i] = *reinterpret_cast<uint32_t*>(&h);
        add_bf16x2(sum[i & 1], pk[i]);
    }
    tmem_st16_async(t_p, pk);
    sum[0] = add2(sum[0], sum[1]);
    return sum[0].x + sum[0].y;
}
// The greater of the two, or NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
// Greatest of 32 scores, NaN if one is.
__device__ __forceinline__ float max32(const uint32_t (&x)[32]) {
    float m[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        m[e] = max_nan(__uint_as_float(x[e]), __uint_as_float(x[e + 4]));
#pragma unroll
        for (int i = 8; i < 32; i += 8)
            m[e] = max_nan(m[e], max_nan(__uint_as_float(x[i + e]), __uint_as_float(x[i + e + 4])));
    }
    return max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3]));
}
// Columns behind `seen` of 32 scores become -inf.
__device__ __forceinline__ void mask32(uint32_t (&x)[32], int seen) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (i > seen) x[i] = 0xff800000u;
}

// One stretch of a share: steps [step, step + n) of an item.  A warp walks through its CTA's share
// item by item; all warps do so alike.
struct Walk {
    int b, tile, head, step, n;
    Seq s;
    int tiles, steps;           // of the sequence; of the item
    long long left;             // steps of the share, this stretch's among them

    __device__ __forceinline__ void enter(const SharePlan& u) {
        steps = share_steps(u, s, tile);
        n = (int)(left < steps - step ? left : steps - step);
    }
    __device__ __forceinline__ void begin(const PagedArgs& p, const SharePlan& u, const ShareStart& st, int index) {
        const long long end = st.share * (index + 1);
        left = (end < st.total ? end : st.total) - st.share * index;
        b = st.b;
        s = load_seq(p, b);
        tiles = share_tiles(u, s);
        locate_step(u, s, p.Hkv, st.off, tile, head, step);
        enter(u);
    }
    __device__ __forceinline__ bool next(const PagedArgs& p, const SharePlan& u) {
        left -= n;
        if (left <= 0) return false;
        step = 0;
        if (++head == p.Hkv) {
            head = 0;
            if (++tile >= tiles) {
                // the next sequence with work, 32 at a time
                tile = 0;
                const int lane = threadIdx.x & 31;
                int b0 = b + 1;
                unsigned hit = 0;
                for (; b0 < p.B; b0 += 32) {
                    Seq t = {0, 0, 0};
                    if (b0 + lane < p.B) t = load_seq(p, b0 + lane);
                    hit = __ballot_sync(0xffffffffu, share_tiles(u, t) > 0);
                    if (hit) {
                        const int src = __ffs(hit) - 1;
                        b = b0 + src;
                        s.q0 = __shfl_sync(0xffffffffu, t.q0, src);
                        s.nq = __shfl_sync(0xffffffffu, t.nq, src);
                        s.kv = __shfl_sync(0xffffffffu, t.kv, src);
                        break;
                    }
                }
                if (!hit) return false;
                tiles = share_tiles(u, s);
            }
        }
        enter(u);
        return true;
    }
};
// What a stretch asks of the stages.
template <int HD>
struct Stretch {
    using S = TcShape<HD>;
    int k_begin, k_end;         // keys [k_begin, k_end)
    int rows[S::STAGES], nh[S::STAGES];     // of each stage: rows, blocks of KH keys
    int blocks, tiles;          // the longest stage's blocks and key tiles

    __device__ __forceinline__ Stretch(const Walk& w, const SharePlan& u) {
        const int row0 = w.tile * u.rt, half = u.rt / S::STAGES, ctx = w.s.kv - w.s.nq;
        k_begin = w.step * STEP_KEYS;
        k_end = 0;
        blocks = 0;
#pragma unroll
        for (int s = 0; s < S::STAGES; ++s) {
            rows[s] = max(0, min(half, w.s.nq * u.g - row0 - s * half));
            int keys = rows[s] > 0 ? ctx + (row0 + s * half + rows[s] - 1) / u.g + 1 : 0;
            if (!u.whole) keys = min(keys, (w.step + w.n) * STEP_KEYS);
            nh[s] = max(0, (keys - k_begin + S::KH - 1) / S::KH);
            k_end = max(k_end, keys);
            // the same in every lane, and known as such: loops over them keep a warp converged
            nh[s] = __shfl_sync(0xffffffffu, nh[s], 0);
            blocks = max(blocks, nh[s]);
        }
        k_end = __shfl_sync(0xffffffffu, k_end, 0);
        tiles = (blocks + S::NB - 1) / S::NB;
    }
    // of a stage that is no compile-time constant
    __device__ __forceinline__ int pick(const int (&v)[S::STAGES], int s) const {
        int x = v[0];
#pragma unroll
        for (int i = 1; i < S::STAGES; ++i) x = s == i ? v[i] : x;
        return x;
    }
};

// A ring position: slot and the parity of its round.
template <int SLOTS>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == SLOTS) {
            slot = 0;
            phase ^= 1;
        }
    }
};

template <int HD>
__global__ void __launch_bounds__(TcShape<HD>::THREADS, TcShape<HD>::CTAS)
k_paged_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmKV, PagedArgs p,
           PagedAttnArgs a, SharePlan u, int q_box_bytes) {
    using S = TcShape<HD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);
    uint64_t* q_empty = q_full + 1;             // an item's last scores are computed
    uint64_t* kv_full = q_empty + 1;            // [SLOTS]
    uint64_t* kv_empty = kv_full + S::SLOTS;    // [SLOTS]
    uint64_t* s_full = kv_empty + S::SLOTS;     // [stage] the next block's scores
    uint64_t* p_full = s_full + S::STAGES;      // [stage] its probabilities, O rescaled
    uint64_t* o_done = p_full + S::STAGES;      // [stage] an item's last product
    uint64_t* tail_full = o_done + S::STAGES;   // [SLOTS] a V tile whose end is to be cleared
    uint64_t* drained = tail_full + S::SLOTS;          // after a timeout: the MMAs issued have completed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
    __shared__ int abort_flag;
    __shared__ ShareSmem share_sm;

    // No wait for the kernel in front here: it is the one that takes this batch's other sequences, it
    // lets this one start only behind its own wait for what came before, and neither reads what the
    // other writes.  The wait stands at the end, so that this kernel's completion covers that one's.
    ShareStart st;
    ShareCut* cut = reinterpret_cast<ShareCut*>(a.part + u.cuts) + blockIdx.x;
    if (!find_share(p, u, blockIdx.x, share_sm, st)) {
        if (!u.whole && threadIdx.x == 0) cut->step = 0;
        pdl_trigger();
        pdl_wait();
        return;
    }
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int half = u.rt / S::STAGES;          // rows per stage: whole tokens

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < S::SLOTS; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 1);
            mbar_init(&tail_full[s], 1);
        }
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_done[i], 1);
        }
        mbar_init(drained, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == S::ISSUER) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(S::TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // behind the allocation, which a kernel that starts early could otherwise get in front of
    pdl_trigger();

    Walk w;
    w.begin(p, u, st, blockIdx.x);
    if (!u.whole && threadIdx.x == 0) *cut = {w.s, w.tile, w.head, w.step, blockIdx.x * st.share - w.step, st.share};
    if (warp < S::SOFTMAX_WARPS) {
        const int s = warp >> 2, r = (warp & 3) * 32 + lane;        // stage, row of the stage
        const uint32_t t_s = tmem + s * S::KH + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t t_o = tmem + S::O_COL + s * HD + ((uint32_t)((warp & 3) * 32) << 16);
        const float c2 = a.scale * LOG2E;
        uint32_t s_phase = 0, o_phase = 0;
        bool ok = true, first = true;
        do {
            const Stretch<HD> x_(w, u);
            const int nh = x_.pick(x_.nh, s);
            const bool mine = r < x_.pick(x_.rows, s), whole = w.n == w.steps;
            const int row = w.tile * u.rt + s * half + r;
            const int slot = 2 * blockIdx.x + (first ? 0 : 1);
            first = false;
            if (nh == 0) continue;
            const int limit = mine ? w.s.kv - w.s.nq + row / u.g - x_.k_begin : -1;    // last key, from the first
            // Where two CTAs share an SM a warp without rows leaves its issue slots to the others; its rows of O
            // hold anything.  (9 turns with heads of 64: 100 -> 98 us; with heads of 128, alone on its SM, 135
            // -> 139 us.)
            const bool idle = S::CTAS > 1 && !__any_sync(0xffffffffu, mine);
            float m = -INFINITY, l = 0.f;       // m of the scaled scores
            for (int h = 0; h < nh; ++h) {
                ok = __all_sync(0xffffffffu, mbar_wait(&s_full[s], s_phase, &abort_flag));
                if (!ok) break;
                s_phase ^= 1;
                if (idle) {
                    if (lane == 0) mbar_arrive(&p_full[s]);
                    continue;
                }
                tc_fence_after();
                const int seen = limit - h * S::KH;         // columns 0 .. seen of this block are seen
                const bool masked = __any_sync(0xffffffffu, seen < S::KH - 1);
                float mx = -INFINITY;
                // Where two CTAs share the registers the scores are read twice, for the maximum and for the
                // exponentials.
                constexpr int KEEP = S::CTAS == 1 ? S::KH / 32 : 2;
                uint32_t x[KEEP][32];
#pragma unroll
                for (int c = 0; c < S::KH / 32; c += KEEP) {
#pragma unroll
                    for (int k = 0; k < KEEP; ++k) tmem_ld32_async(t_s + 32 * (c + k), x[k]);
#pragma unroll
                    for (int k = 0; k < KEEP; ++k) {
                        tmem_wait_ld(x[k]);
                        if (masked) mask32(x[k], seen - 32 * (c + k));
                        mx = max_nan(mx, max32(x[k]));
                    }
                }
                mx *= c2;
                // (a first maximum needs no rescale: the first product overwrites O, and l is 0)
                const bool grow = !(mx <= m + RESCALE) || m == -INFINITY;
                if (__any_sync(0xffffffffu, grow)) {
                    // A score that is NaN, or +inf (inf - inf is NaN), makes the row NaN from here on: the
                    // polynomial's clamp would lose it.
                    const float to = mx == INFINITY ? __int_as_float(0x7fffffff) : grow ? mx : m;
                    const float al = m == -INFINITY ? 1.f : ex2_approx(m - to);
                    l *= al;
                    m = to;
                    if (h > 0) {
#pragma unroll 1
                        for (int c = 0; c < HD; c += 32) {
                            float ov[32];
                            tmem_ld32(t_o + c, ov);
#pragma unroll
                            for (int i = 0; i < 32; ++i) ov[i] *= al;
                            tmem_st32(t_o + c, ov);
                        }
                    }
                }
                const float neg = m == -INFINITY ? 0.f : -m;        // a row that has seen nothing yet
                // where columns are masked every exponential is exact at -inf
#pragma unroll
                for (int c = 0; c < S::KH / 32; ++c) {
                    if (S::CTAS > 1) {
                        tmem_ld32_async(t_s + 32 * c, x[0]);
                        tmem_wait_ld(x[0]);
                        if (masked) mask32(x[0], seen - 32 * c);
                    }
                    const uint32_t(&xc)[32] = x[S::CTAS > 1 ? 0 : c];
                    l += masked ? softmax32<0>(xc, t_s + 16 * c, c2, neg) : softmax32<S::POLY>(xc, t_s + 16 * c, c2, neg);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[s]);
            }
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&o_done[s], o_phase, &abort_flag));
            if (!ok) break;
            o_phase ^= 1;
            // (the next item's first product waits for probabilities that come behind these reads)
            tc_fence_after();
            if (!whole) {
                float* pr = share_part(a, u, slot, HD) + s * half + r;
#pragma unroll 1
                for (int c = 0; c < HD; c += 32) {
                    float ov[32];
                    tmem_ld32(t_o + c, ov);
                    if (mine) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) pr[(c + i) * u.rt] = ov[i];
                    }
                }
                if (mine) {
                    pr[HD * u.rt] = m;
                    pr[(HD + 1) * u.rt] = l;
                }
            } else {
                const float inv = 1.0f / l;
                bf16* o = reinterpret_cast<bf16*>(a.o) + (long long)(w.s.q0 + row / u.g) * a.o_stride +
                          (long long)(w.head * u.g + row % u.g) * HD;
#pragma unroll 1
                for (int c = 0; c < HD; c += 32) {
                    float ov[32];
                    tmem_ld32(t_o + c, ov);
#pragma unroll
                    for (int i = 0; i < 32; ++i) ov[i] *= inv;
                    if (mine) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8) st16(o + c + i, Vec16<bf16>::pack(ov + i));
                    }
                }
            }
        } while (w.next(p, u));
        if (!ok) {
            abort_flag = 1;
            if (lane == 0) raise_flag(p.hdr, ERR_TIMEOUT);
        }
    } else {
        if (warp == S::PRODUCER) {
            // lane i loads atom i % ATOMS of page i / ATOMS of a tile
            const int page_rows = min(KT, 1 << p.page_shift);
            const int pg = lane / S::ATOMS, atom = lane % S::ATOMS;
            Ring<S::SLOTS> ring;
            uint32_t q_phase = 0, items = 0, tail_phases = 0, tails = 0;     // bits of slots: phases, last item a tail
            bool ok = true;
            do {
                const Stretch<HD> x_(w, u);
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(q_empty, q_phase ^ 1, &abort_flag)))) break;
                int boxes_q = 0;
#pragma unroll
                for (int s = 0; s < S::STAGES; ++s) boxes_q += x_.nh[s] > 0;
                if (lane == 0) mbar_expect_tx(q_full, boxes_q * q_box_bytes);
                __syncwarp();
                if (lane < S::STAGES * S::ATOMS && x_.pick(x_.nh, pg) > 0)
                    tma_load_3d(smem + pg * S::Q_BYTES + atom * 128 * 128, &tmQ, q_full, 64 * atom, w.head * u.g,
                                w.s.q0 + w.tile * u.toks + pg * (u.toks / S::STAGES));
                q_phase ^= 1;
                for (int j = 0; j < x_.tiles && ok; ++j) {
                    const int have = x_.k_end - x_.k_begin - j * KT;        // keys from this tile on
                    const int key = x_.k_begin + j * KT + pg * page_rows;
                    const bool mine = pg * page_rows < min(KT, have);
                    const int boxes = min(KT / page_rows, (have + page_rows - 1) / page_rows) * S::ATOMS;
                    const int page = mine ? max(load_page(p, w.b, key), 0) : 0;
                    const int in_page = key & ((1 << p.page_shift) - 1);
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv) {
                        ok = __all_sync(0xffffffffu, mbar_wait(&kv_empty[ring.slot], ring.phase ^ 1, &abort_flag));
                        if (!ok) break;
                        uint8_t* tile = smem + S::OFF_KV + ring.slot * S::T_BYTES;
                        // (an item's last V tile may end inside: the clearing warp hands it on)
                        const bool tail = kv == 1 && have < KT;
                        uint64_t* bar = tail ? &tail_full[ring.slot] : &kv_full[ring.slot];
                        if (lane == 0) mbar_expect_tx(bar, boxes * page_rows * 128);
                        __syncwarp();
                        if (mine)
                            tma_load_2d(tile + atom * KT * 128 + pg * page_rows * 128, &tmKV, bar, 64 * atom,
                                        (((page * 2 + kv) * p.Hkv + w.head) << p.page_shift) + in_page);
                        tail_phases ^= (tail ? 1u : 0u) << ring.slot;
                        tails = (tails & ~(1u << ring.slot)) | (tail ? 1u : 0u) << ring.slot;
                        ring.next();
                        ++items;
                    }
                }
                if (!ok) break;
            } while (w.next(p, u));
            if (!ok) {
                abort_flag = 1;
                // the copies in flight land before the shared memory is given back
                if (lane == 0) {
                    mbar_wait(q_full, q_phase ^ 1, nullptr);
                    for (int i = 0; i < S::SLOTS && i < (int)items; ++i) {
                        // the slot's last round: behind the ring's position it is the round before
                        const uint32_t ph = i < ring.slot ? ring.phase : ring.phase ^ 1;
                        if (tails >> i & 1) mbar_wait(&tail_full[i], (tail_phases >> i & 1) ^ 1, nullptr);
                        else mbar_wait(&kv_full[i], ph, nullptr);
                    }
                }
            }
        } else if (warp == S::CLEARER) {
            // Slots behind a sequence's last key hold anything, and 0 * NaN is NaN: in the last V tile of an
            // item that ends inside they become zeros before the tile is handed on.
            int slot = 0;
            uint32_t phases = 0;
            bool ok = true;
            do {
                const Stretch<HD> x_(w, u);
                const int have = x_.k_end - x_.k_begin - (x_.tiles - 1) * KT;
                slot = (slot + 2 * x_.tiles - 1) % S::SLOTS;
                if (have < KT) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&tail_full[slot], phases >> slot & 1, &abort_flag));
                    if (!ok) break;
                    phases ^= 1u << slot;
                    uint8_t* tile = smem + S::OFF_KV + slot * S::T_BYTES;
                    for (int i = lane; i < (KT - have) * S::ATOMS * 8; i += 32) {
                        const int piece = i & 7, at = (i >> 3) % S::ATOMS, r = have + (i >> 3) / S::ATOMS;
                        *reinterpret_cast<uint4*>(tile + at * KT * 128 + r * 128 + piece * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&kv_full[slot]);
                }
                slot = (slot + 1) % S::SLOTS;
            } while (w.next(p, u));
            if (!ok) abort_flag = 1;
        } else {
            constexpr uint32_t id_s = idesc_bf16(128, S::KH), id_o = idesc_bf16(128, HD) | IDESC_B_MN;
            Ring<S::SLOTS> ring;
            uint32_t q_phase = 0, p_phase[S::STAGES] = {};
            bool ok = true;
            auto commit = [&](uint64_t* bar) {
                if (elect_one()) umma_commit(bar);
                __syncwarp();
            };
            auto wait_kv = [&](const Ring<S::SLOTS>& at) {
                return __all_sync(0xffffffffu, mbar_wait(&kv_full[at.slot], at.phase, &abort_flag));
            };
            auto issue_s = [&](int s, int b, int slot) {    // S_s = Q_s K^T, block b of the K tile in `slot`
                const uint64_t dq0 = sdesc_sw128(smem + s * S::Q_BYTES);
                const uint64_t dk0 = sdesc_sw128(smem + S::OFF_KV + slot * S::T_BYTES + b * S::KH * 128);
                if (elect_one()) {
#pragma unroll
                    for (int at = 0; at < S::ATOMS; ++at)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma(tmem + s * S::KH, dq0 + at * (128 * 128 >> 4) + 2 * k, dk0 + at * (KT * 128 >> 4) + 2 * k,
                                 id_s, (at | k) != 0);
                    umma_commit(&s_full[s]);
                }
                __syncwarp();
            };
            do {
                const Stretch<HD> x_(w, u);
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(q_full, q_phase, &abort_flag)))) break;
                q_phase ^= 1;
                Ring<S::SLOTS> k = ring;                    // K of tile j
                if (!(ok = wait_kv(k))) break;
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < S::STAGES; ++s)
                    if (x_.nh[s] > 0) issue_s(s, 0, k.slot);
                if (S::NB == 1) commit(&kv_empty[k.slot]);
                if (x_.blocks == 1) commit(q_empty);
                for (int j = 0; j < x_.tiles && ok; ++j) {
                    ring.next();
                    const Ring<S::SLOTS> v = ring;
                    ring.next();
                    const bool more = j + 1 < x_.tiles;
                    if (!(ok = wait_kv(v))) break;
#pragma unroll
                    for (int b = 0; b < S::NB; ++b) {
                        const int h = j * S::NB + b;
                        // the block behind this one is in the same K tile, or the first of the next
                        if (b + 1 == S::NB) {
                            k = ring;
                            if (more && !(ok = ok && wait_kv(k))) continue;
                        }
                        const uint64_t dv = sdesc_mn_sw128(smem + S::OFF_KV + v.slot * S::T_BYTES + b * S::KH * 128, KT * 128);
#pragma unroll
                        for (int s = 0; s < S::STAGES; ++s) {
                            if (h >= x_.nh[s] || !ok) continue;
                            ok = __all_sync(0xffffffffu, mbar_wait(&p_full[s], p_phase[s], &abort_flag));
                            if (!ok) continue;
                            p_phase[s] ^= 1;
                            tc_fence_after();
                            if (elect_one()) {
#pragma unroll
                                for (int i = 0; i < S::KH / 16; ++i)
                                    umma_ta(tmem + S::O_COL + s * HD, tmem + s * S::KH + i * 8, dv + i * (16 * 128 >> 4), id_o,
                                            (h | i) != 0);
                                if (h + 1 == x_.nh[s]) umma_commit(&o_done[s]);
                            }
                            __syncwarp();
                            if (h + 1 < x_.nh[s]) issue_s(s, (b + 1) % S::NB, k.slot);
                        }
                        // the K tile's last block of scores is issued
                        if (ok && (S::NB == 1 ? more : b + 2 == S::NB)) commit(&kv_empty[k.slot]);
                        if (ok && h + 2 == x_.blocks) commit(q_empty);
                    }
                    if (ok) commit(&kv_empty[v.slot]);
                }
                if (!ok) break;
            } while (w.next(p, u));
            if (!ok) {
                abort_flag = 1;
                if (elect_one()) {
                    umma_commit(drained);
                    mbar_wait(drained, 0, nullptr);
                }
                __syncwarp();
            }
        }
    }
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    if (warp == S::ISSUER) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::TMEM_COLS));
    }
}

template <int HD>
cudaError_t run(Launch L, const PagedArgs& p, const PagedAttnArgs& a, const SharePlan& u) {
    using S = TcShape<HD>;
    cudaError_t e = cudaFuncSetAttribute(k_paged_tc<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    const int toks = u.toks / S::STAGES;        // tokens per stage
    CUtensorMap tq, tkv;
    const uint64_t qdims[3] = {(uint64_t)HD, (uint64_t)a.H, (uint64_t)p.N};
    const uint64_t qstr[2] = {(uint64_t)HD * 2, (uint64_t)a.q_stride * 2};
    const uint32_t qbox[3] = {64, (uint32_t)u.g, (uint32_t)toks};
    const uint64_t kvdims[2] = {(uint64_t)HD, ((uint64_t)p.n_pages * 2 * p.Hkv) << p.page_shift};
    const uint64_t kvstr[1] = {(uint64_t)HD * 2};
    const uint32_t page = 1u << p.page_shift;
    const uint32_t kvbox[2] = {64, page < KT ? page : KT};
    if (!tma_map_bf16_new(&tq, a.q, 3, qdims, qstr, qbox) || !tma_map_bf16_new(&tkv, a.pool, 2, kvdims, kvstr, kvbox))
        return cudaErrorInvalidValue;
    return launch_k(L, k_paged_tc<HD>, (unsigned)u.ctas, S::THREADS, S::SMEM, tq, tkv, p, a, u, u.g * toks * 128 * S::ATOMS);
}

}  // namespace

cudaError_t launch_paged_tc(Launch L, const PagedArgs& p, const PagedAttnArgs& a, const SharePlan& u) {
    return a.hd == 64 ? run<64>(L, p, a, u) : run<128>(L, p, a, u);
}

}  // namespace rlt
