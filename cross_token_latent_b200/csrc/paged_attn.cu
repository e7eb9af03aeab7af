// Causal attention of new tokens over a paged key/value cache: row r (token i of sequence b, at
// position t) reads keys 0 .. t of its sequence, query head j those of key head j / g.
//
// One pass over the keys with the running maximum and sum of the softmax.  Rows of one key head's
// group are taken together (rows are numbered i * g + j), so that shared keys are read once; a
// long key axis is cut into units (paged.cuh) whose partial states k_paged_join merges.
#include "paged.cuh"
#include "sm100.cuh"

namespace rlt {

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float NEG_BIG = -1e30f;

// One output row of a cut item from n partial states, by a block of 128 threads; state j's row is at
// states + j * stride.  128 states at a time: a thread per state looks at its maximum and sum, then
// threads over the columns (and over the states, where a row has fewer columns than there are
// threads) add them up.
constexpr int JOIN_THREADS = 128;
template <typename T>
__device__ __forceinline__ void join_row(T* o, int hd, int n, const float* __restrict__ states, long long stride) {
    __shared__ float weight[JOIN_THREADS], top[4], sums[4], acc_sm[JOIN_THREADS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int col = tid % hd, part = tid / hd, parts = JOIN_THREADS / hd;
    float m = NEG_BIG, l = 0.f, acc = 0.f;
    for (int j0 = 0; j0 < n; j0 += JOIN_THREADS) {
        const int here = min(JOIN_THREADS, n - j0);
        float2 ml = make_float2(NEG_BIG, 0.f);
        const float* now = states + j0 * stride;
        if (tid < here) ml = *reinterpret_cast<const float2*>(now + tid * stride + hd);
        const float mw = warp_max(ml.x);
        if (lane == 0) top[warp] = mw;
        __syncthreads();
        const float to = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
        const float w = exp2f(ml.x - to), old = exp2f(m - to);
        weight[tid] = w;
        const float lw = warp_sum(w * ml.y);
        if (lane == 0) sums[warp] = lw;
        __syncthreads();
        l = l * old + ((sums[0] + sums[1]) + (sums[2] + sums[3]));
        acc *= old;
        m = to;
        for (int j = part; j < here; j += 8 * parts) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = j + k * parts < here ? now[(j + k * parts) * stride + col] : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) acc = fmaf(j + k * parts < here ? weight[j + k * parts] : 0.f, v[k], acc);
        }
        __syncthreads();                        // the weights are read
    }
    acc_sm[tid] = acc;
    __syncthreads();
    if (part == 0) {
        for (int i = 1; i < parts; ++i) acc += acc_sm[i * hd + col];
        o[col] = from_f<T>(acc / l);
    }
}

// Joins the partial states of the cut items.  The first n1 blocks of x are cut items of the plan u,
// whose rows the first y1 blocks of y take in turn.  With the plan us, block n1 + c - 1 is the item that
// share c begins inside of, if share c is the first to: 128 rows, a thread each, of 16 columns (y: column
// and row blocks; 9 turns with heads of 64 take 98 us in all with 8 columns, 95 with 16, 96 with 32).
constexpr int JOIN_COLS = 16;
template <typename T>
__global__ void __launch_bounds__(JOIN_THREADS) k_paged_join(PagedArgs p, PagedAttnArgs a, UnitPlan u, int n1,
                                                             int y1, SharePlan us) {
    if ((int)blockIdx.x < n1) {
        // The kernel in front waited for its predecessor before it let this one start, so the batch's
        // lengths may be read here; the partial states only behind the wait.
        Unit w;
        const bool any = (int)blockIdx.y < y1 && find_unit(p, u, blockIdx.x, true, w);
        pdl_wait();
        pdl_trigger();
        if (!any) return;
        const int row0 = w.tile * u.rt, rows = min(u.rt, w.s.nq * u.g - row0);
        for (int i = blockIdx.y; i < rows; i += y1) {
            const int tok = (row0 + i) / u.g, keys = w.s.kv - w.s.nq + tok + 1;
            const int n = min(w.n_splits, (keys + w.chunk - 1) / w.chunk);      // units that saw a key of this row
            T* o = reinterpret_cast<T*>(a.o) + (w.s.q0 + tok) * a.o_stride +
                   (long long)(w.head * u.g + (row0 + i) % u.g) * a.hd;
            join_row(o, a.hd, n, part_row(a, u, w.slot, i, a.hd), (long long)u.rt * (a.hd + 2));
            __syncthreads();                    // its shared memory is free
        }
        return;
    }
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x - n1 + 1;
    const ShareCut cut = reinterpret_cast<const ShareCut*>(a.part + us.cuts)[c];
    if (cut.step == 0) return;
    const int c0 = (int)(cut.begin / cut.share), row0 = cut.tile * us.rt;
    const int cols = a.hd / JOIN_COLS, i = blockIdx.y / cols * JOIN_THREADS + threadIdx.x, col = blockIdx.y % cols * JOIN_COLS;
    if (c0 != c - 1 || i >= us.rt || row0 + i >= cut.s.nq * us.g) return;
    const int tok = (row0 + i) / us.g;
    // shares up to the step of the row's last key
    const int n = (int)((cut.begin + (cut.s.kv - cut.s.nq + tok) / STEP_KEYS) / cut.share) - c0 + 1;
    // a share that begins with the item, or inside it, has it in its first slot
    const int first = 2 * c0 + (cut.begin != c0 * cut.share ? 1 : 0);
    float m = NEG_BIG, l = 0.f, acc[JOIN_COLS];
#pragma unroll
    for (int k = 0; k < JOIN_COLS; ++k) acc[k] = 0.f;
    constexpr int AHEAD = 2;                    // states whose loads are in flight together
    for (int j0 = 0; j0 < n; j0 += AHEAD) {
        float v[AHEAD][JOIN_COLS], mj[AHEAD], lj[AHEAD];
        float to = m;
#pragma unroll
        for (int b = 0; b < AHEAD; ++b) {
            const int j = min(j0 + b, n - 1);
            const float* x = share_part(a, us, j == 0 ? first : 2 * (c0 + j), a.hd) + i;
#pragma unroll
            for (int k = 0; k < JOIN_COLS; ++k) v[b][k] = x[(col + k) * us.rt];
            mj[b] = j0 + b < n ? x[a.hd * us.rt] : NEG_BIG;
            lj[b] = x[(a.hd + 1) * us.rt];
        }
#pragma unroll
        for (int b = 0; b < AHEAD; ++b) to = fmaxf(to, mj[b]);
        const float old = exp2f(m - to);
        m = to;
        l *= old;
#pragma unroll
        for (int k = 0; k < JOIN_COLS; ++k) acc[k] *= old;
#pragma unroll
        for (int b = 0; b < AHEAD; ++b) {
            const float f = exp2f(mj[b] - to);
            l = fmaf(lj[b], f, l);
#pragma unroll
            for (int k = 0; k < JOIN_COLS; ++k) acc[k] = fmaf(v[b][k], f, acc[k]);
        }
    }
    const float inv = 1.0f / l;
    T* o = reinterpret_cast<T*>(a.o) + (cut.s.q0 + tok) * a.o_stride +
           (long long)(cut.head * us.g + (row0 + i) % us.g) * a.hd + col;
#pragma unroll
    for (int k = 0; k < JOIN_COLS; ++k) acc[k] *= inv;
#pragma unroll
    for (int k = 0; k < JOIN_COLS; k += Vec16<T>::N) st16(o + k, Vec16<T>::pack(acc + k));
}

// ------------------------------------------------------------------ few rows, tensor cores
// 16 rows of one key head against groups of keys that the warps take in turn, on mma.m16n8k16.
// What bounds it is reading the keys and values once; a tile's 16 rows are mostly empty in a decode
// step, and the warp-level product needs no tensor memory and no barrier between warps on the way.
// 16 keys lie in one page, side by side, and their values again, so each warp has them copied whole
// (cp.async.bulk) into a ring of its own, groups ahead; loading the fragments straight from memory
// left too few bytes in flight beside the accumulators (64 ragged contexts, 1.1 GB: 220 us, 77 % of
// the copy rate).  Narrow heads take several 16 keys per group, which share one look at the maximum.
//
// The contraction over head_dim may run in any order, so lane t of a quad takes 8 consecutive
// elements of its key (16 bytes) and the queries are loaded to match; columns of the output are
// dealt so that a lane reads 16 consecutive bytes of a value and ends up with consecutive output
// columns.
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// W consecutive 32-bit words
template <int W>
__device__ __forceinline__ void load_words(const void* p, uint32_t* r) {
    if (W == 1) r[0] = *reinterpret_cast<const uint32_t*>(p);
    if (W == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        r[0] = x.x; r[W > 1 ? 1 : 0] = x.y;
    }
    if (W == 4) {
        const uint4 x = ld16(p);
        r[0] = x.x; r[W > 1 ? 1 : 0] = x.y; r[W > 2 ? 2 : 0] = x.z; r[W > 2 ? 3 : 0] = x.w;
    }
}

constexpr int MMA_WARPS = 4;
template <int HD>
struct MmaShape {
    static constexpr int QW = HD >= 32 ? 4 : 2;             // words per lane and piece of a key
    static constexpr int QP = HD >= 32 ? HD / 32 : 1;       // pieces
    static constexpr int VW = HD >= 64 ? 4 : HD / 16;       // words per lane and piece of a value
    static constexpr int VP = HD >= 64 ? HD / 64 : 1;
    static constexpr int NT = HD / 8;                       // output tiles of 8 columns
    static constexpr int LD = HD + 4;
    static constexpr int M = HD == 128 ? 1 : (HD == 64 ? 2 : 4);    // blocks of 16 keys in a group
    static constexpr int BLOCK = 16 * HD * 2;               // bytes of a block's keys, and of its values
    static constexpr int GROUP = M * 2 * BLOCK;             // [block][keys, values]
    // Stages of a warp's ring, CTAs per SM: 192 KB in flight at head widths of 128 and 64.  (At 128, two
    // CTAs with three stages take 193 us for the 64 contexts where three with two take 182 us.)
    static constexpr int STAGES = 2;
    static constexpr int CTAS = HD >= 64 ? 3 : 4;
    static constexpr int RING = MMA_WARPS * STAGES * GROUP;
    static constexpr int JOIN = MMA_WARPS * 16 * LD * 4;    // over the rings, when they are through
    static constexpr int SMEM = RING > JOIN ? RING : JOIN;
};

// (Narrow heads are bound by the instructions per key: 100 contexts of 500 to 8000 keys, 16 heads of 16, take
// 132 us, half the copy rate, at 64 % issue.  Chunks read all keys again for every 16 rows, from L2: a prompt of
// 2000 tokens takes 60 us with 16 heads of 32 and 44 us with heads of 16, 52 % issue.)
template <int HD>
__global__ void __launch_bounds__(MMA_WARPS * 32, MmaShape<HD>::CTAS) k_paged_mma(PagedArgs p, PagedAttnArgs a, UnitPlan u,
                                                                                  int units) {
    using S = MmaShape<HD>;
    extern __shared__ __align__(128) uint8_t ring_sm[];     // [warps][STAGES][keys, values]
    float* sm = reinterpret_cast<float*>(ring_sm);          // [warps][16][LD]: accumulators, maximum, sum
    __shared__ uint64_t full[MMA_WARPS][S::STAGES];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    if (lane == 0) {
        for (int i = 0; i < S::STAGES; ++i) mbar_init(&full[warp][i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    pdl_wait();
    pdl_trigger();
    uint8_t* ring = ring_sm + warp * S::STAGES * S::GROUP;
    int stage = 0;                                          // of the next group to be computed
    uint32_t phase = 0;
    const float c2 = a.scale * LOG2E;
    const bf16* pool = reinterpret_cast<const bf16*>(a.pool);
    const long long head_elems = (long long)HD << p.page_shift, v_off = p.Hkv * head_elems;
    const int page_mask = (1 << p.page_shift) - 1;

    for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
        Unit w;
        if (!find_unit(p, u, unit, false, w)) return;
        const int row0 = w.tile * 16, rows = min(16, w.s.nq * u.g - row0), ctx = w.s.kv - w.s.nq;
        const int last = ctx + (row0 + rows - 1) / u.g;
        const int k_begin = w.split * w.chunk, k_end = min(last + 1, k_begin + w.chunk);
        if (k_begin >= k_end) continue;

        // this warp's groups: 16 M keys from k_begin + 16 M (warp + 4 i); lane j keeps the page of block
        // b0 + j, blocks counted through the warp's groups
        constexpr int KG = 16 * S::M;
        const int n_groups = (k_end - k_begin + KG - 1) / KG;
        const int mine = n_groups > warp ? (n_groups - warp + MMA_WARPS - 1) / MMA_WARPS : 0;
        auto key0 = [&](int i) { return k_begin + KG * (warp + MMA_WARPS * i); };
        int pages = 0, fill = stage;                        // fill: stage of the next group to be copied
        auto copy = [&](int i) {
            if ((i * S::M & 31) == 0) {
                const int at = key0(i + lane / S::M) + lane % S::M * 16;
                pages = at < k_end ? max(load_page(p, w.b, at), 0) : 0;
            }
            const int m = lane % S::M, key = key0(i) + 16 * m;
            const int page = __shfl_sync(0xffffffffu, pages, (i * S::M + m) & 31);
            if (lane == 0) mbar_expect_tx(&full[warp][fill], min(S::M, (k_end - key0(i) + 15) / 16) * 2 * S::BLOCK);
            __syncwarp();
            if (lane < S::M && key < k_end) {
                const bf16* src = pool + ((long long)page * 2 * p.Hkv + w.head) * head_elems + (long long)(key & page_mask) * HD;
                uint8_t* dst = ring + fill * S::GROUP + m * 2 * S::BLOCK;
                bulk_load(dst, src, S::BLOCK, &full[warp][fill]);
                bulk_load(dst + S::BLOCK, src + v_off, S::BLOCK, &full[warp][fill]);
            }
            if (++fill == S::STAGES) fill = 0;
        };
        for (int i = 0; i < S::STAGES && i < mine; ++i) copy(i);

        uint32_t q[2][S::QP][S::QW];
        int limit[2];                                       // the last key of rows g and g + 8
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = row0 + g + 8 * i, tok = row / u.g;
            const bool ok = g + 8 * i < rows;
            limit[i] = ok ? ctx + tok : -1;
            const bf16* qp = reinterpret_cast<const bf16*>(a.q) + (long long)(w.s.q0 + tok) * a.q_stride +
                             (long long)(w.head * u.g + row % u.g) * HD;
#pragma unroll
            for (int c = 0; c < S::QP; ++c) {
#pragma unroll
                for (int e = 0; e < S::QW; ++e) q[i][c][e] = 0;
                if (ok) load_words<S::QW>(qp + (c * 4 + t) * S::QW * 2, q[i][c]);
            }
        }

        float m[2] = {NEG_BIG, NEG_BIG}, l[2] = {0.f, 0.f};     // m of the scores as they are
        float o[S::NT][4];
#pragma unroll
        for (int j = 0; j < S::NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;

        bool ok = true;
        for (int i = 0; i < mine; ++i) {
            ok = __all_sync(0xffffffffu, mbar_wait(&full[warp][stage], phase, nullptr));
            if (!ok) break;
            const uint8_t* kb = ring + stage * S::GROUP;
            float s[S::M][2][4];
#pragma unroll
            for (int b = 0; b < S::M; ++b)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[b][n][e] = 0.f;
#pragma unroll
            for (int c = 0; c < S::QP; ++c)
#pragma unroll
                for (int b = 0; b < S::M; ++b) {
                    uint32_t kf[2][S::QW];
#pragma unroll
                    for (int n = 0; n < 2; ++n)
                        load_words<S::QW>(kb + b * 2 * S::BLOCK + (8 * n + g) * HD * 2 + (c * 4 + t) * S::QW * 4, kf[n]);
#pragma unroll
                    for (int h = 0; h < S::QW; h += 2) {
                        const uint32_t af[4] = {q[0][c][h], q[1][c][h], q[0][c][h + 1], q[1][c][h + 1]};
#pragma unroll
                        for (int n = 0; n < 2; ++n) mma16816(s[b][n], af, kf[n][h], kf[n][h + 1]);
                    }
                }
            const int k0 = key0(i);
            float mx[2] = {m[0], m[1]};
#pragma unroll
            for (int b = 0; b < S::M; ++b)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (k0 + 16 * b + 8 * n + 2 * t + (e & 1) > limit[e >> 1]) s[b][n][e] = -INFINITY;
                        mx[e >> 1] = fmaxf(mx[e >> 1], s[b][n][e]);
                    }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
                mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            }
            if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float al = ex2_approx((m[r] - mx[r]) * c2);
                    l[r] *= al;
                    m[r] = mx[r];
#pragma unroll
                    for (int j = 0; j < S::NT; ++j) { o[j][2 * r] *= al; o[j][2 * r + 1] *= al; }
                }
            }
            const float mc[2] = {m[0] == NEG_BIG ? 0.f : m[0] * c2, m[1] == NEG_BIG ? 0.f : m[1] * c2};
#pragma unroll
            for (int b = 0; b < S::M; ++b) {
                // probabilities rounded to bf16 for the product; the sum is of the rounded values, so that
                // the result stays a weighted mean of the values
                uint32_t pf[4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        __nv_bfloat162 h = __floats2bfloat162_rn(ex2_approx(fmaf(s[b][n][2 * r], c2, -mc[r])),
                                                                 ex2_approx(fmaf(s[b][n][2 * r + 1], c2, -mc[r])));
                        const uint32_t x = *reinterpret_cast<uint32_t*>(&h);
                        l[r] += __uint_as_float(x << 16) + __uint_as_float(x & 0xffff0000u);
                        pf[2 * n + r] = x;
                    }
                const uint8_t* vb = kb + b * 2 * S::BLOCK + S::BLOCK;
                const int kb0 = k0 + 16 * b;
#pragma unroll
                for (int c = 0; c < S::VP; ++c) {
                    uint32_t vf[4][S::VW];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const int j = 2 * t + (n & 1) + 8 * (n >> 1);       // keys 2t, 2t + 1, 2t + 8, 2t + 9
                        load_words<S::VW>(vb + j * HD * 2 + (c * 8 + g) * S::VW * 4, vf[n]);
                        if (kb0 + 16 > k_end) {
                            // slots behind the last key hold anything, and 0 * NaN is NaN
#pragma unroll
                            for (int e = 0; e < S::VW; ++e) vf[n][e] = kb0 + j < k_end ? vf[n][e] : 0u;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < S::VW; ++e) {
                        mma16816(o[(c * S::VW + e) * 2], pf, __byte_perm(vf[0][e], vf[1][e], 0x5410),
                                 __byte_perm(vf[2][e], vf[3][e], 0x5410));
                        mma16816(o[(c * S::VW + e) * 2 + 1], pf, __byte_perm(vf[0][e], vf[1][e], 0x7632),
                                 __byte_perm(vf[2][e], vf[3][e], 0x7632));
                    }
                }
            }
            __syncwarp();                                   // the stage is read
            if (++stage == S::STAGES) {
                stage = 0;
                phase ^= 1;
            }
            if (i + S::STAGES < mine) copy(i + S::STAGES);
        }
        if (!ok && lane == 0) {
            raise_flag(p.hdr, ERR_TIMEOUT);
            // the copies in flight land before the shared memory is given back
            for (int i = 0; i < S::STAGES; ++i) {
                if (mine > i) mbar_wait(&full[warp][stage], phase, nullptr);
                if (++stage == S::STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }

        // Join the warps.  Lane t of quad g has, of piece c, columns (c * 8 + 2t) * 2 VW .. + 4 VW - 1:
        // tile j's element 0 is column (c * 8 + 2t) * 2 VW + j, element 1 is 2 VW further.
        if (__syncthreads_or(!ok)) return;                  // (behind it the rings are through)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            float* dst = sm + (warp * 16 + g + 8 * r) * S::LD;
            if (g + 8 * r < rows) {
#pragma unroll
                for (int c = 0; c < S::VP; ++c)
#pragma unroll
                    for (int e = 0; e < 2 * S::VW; ++e) {
                        dst[(c * 8 + 2 * t) * 2 * S::VW + e] = o[c * S::VW * 2 + e][2 * r];
                        dst[(c * 8 + 2 * t + 1) * 2 * S::VW + e] = o[c * S::VW * 2 + e][2 * r + 1];
                    }
                if (t == 0) { dst[HD] = m[r] * c2; dst[HD + 1] = l[r]; }
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < rows * HD; i += MMA_WARPS * 32) {
            const int r = i / HD, col = i % HD;
            float mt = NEG_BIG;
#pragma unroll
            for (int x = 0; x < MMA_WARPS; ++x) mt = fmaxf(mt, sm[(x * 16 + r) * S::LD + HD]);
            float lt = 0.f, acc = 0.f;
#pragma unroll
            for (int x = 0; x < MMA_WARPS; ++x) {
                const float* src = sm + (x * 16 + r) * S::LD;
                const float f = ex2_approx(src[HD] - mt);
                lt += f * src[HD + 1];
                acc += f * src[col];
            }
            if (w.n_splits > 1) {
                float* pr = part_row(a, u, w.slot, r, HD);
                pr[col] = acc;
                if (col == 0) { pr[HD] = mt; pr[HD + 1] = lt; }
            } else {
                const int row = row0 + r;
                reinterpret_cast<bf16*>(a.o)[(long long)(w.s.q0 + row / u.g) * a.o_stride +
                                             (long long)(w.head * u.g + row % u.g) * HD + col] = from_f<bf16>(acc / lt);
            }
        }
        fence_proxy_async_smem();                           // the next unit's copies come behind these accesses
        __syncthreads();
    }
}

// ------------------------------------------------------------------ float32
// 8 rows of one key head against groups of 16 keys, every warp on its own as above, on the CUDA cores
// in float32 throughout (the tensor cores would need every operand split into several terms of their
// formats, and a product for each pair of them: not tried).  Lane
// 16 j + k scores key k for rows 4 j .. 4 j + 3 and then has columns k, k + 16, .. of the output of
// those rows, the probabilities going round by shared memory.  Scoring, the four elements of a key that a
// lane takes next are the (step + key)-th: side by side, keys lie HD floats apart, and lanes that all
// took the same would meet in the same banks.  What bounds it is a warp's chain per
// 16 keys (wait, scores, maximum, exponentials, products): 6 chunks with heads of 16 take 22.6 us at 16 % of the
// multiply-add pipe and 36 % issue; a decode step of 240 contexts with 8 heads of 64 takes 288 us, half the
// measured copy rate, at 51 % issue, seven of eight rows of a tile being empty.
template <int HD>
struct F32Shape {
    static constexpr int RT = 8;
    static constexpr int LD = HD + 4;
    static constexpr int BLOCK = 16 * HD * 4;               // bytes of a group's keys, and of its values
    static constexpr int STAGES = 2;
    static constexpr int CTAS = HD == 128 ? 1 : (HD == 64 ? 3 : 5);
    static constexpr int RING = MMA_WARPS * STAGES * 2 * BLOCK;
    static constexpr int JOIN = MMA_WARPS * RT * LD * 4;    // over the rings, when they are through
    static constexpr int ROWS = RT * HD * 4;                // the queries, behind them
    static constexpr int SMEM = (RING > JOIN ? RING : JOIN) + ROWS;
};

template <int HD>
__global__ void __launch_bounds__(MMA_WARPS * 32, F32Shape<HD>::CTAS) k_paged_f32(PagedArgs p, PagedAttnArgs a, UnitPlan u) {
    using S = F32Shape<HD>;
    constexpr int NC = HD / 16, NP = HD / 4;                // columns per lane, 16-byte pieces of a key
    extern __shared__ __align__(128) uint8_t ring_sm[];     // [warps][STAGES][keys, values]
    float* sm = reinterpret_cast<float*>(ring_sm);          // [warps][RT][LD]: accumulators, maximum, sum
    float* qs = reinterpret_cast<float*>(ring_sm + S::SMEM - S::ROWS);
    __shared__ __align__(16) float ps[MMA_WARPS][S::RT][16];        // probabilities of a warp's group
    __shared__ uint64_t full[MMA_WARPS][S::STAGES];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = lane >> 4, k = lane & 15;
    if (lane == 0) {
        for (int i = 0; i < S::STAGES; ++i) mbar_init(&full[warp][i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    pdl_wait();
    pdl_trigger();
    Unit w;
    if (!find_unit(p, u, blockIdx.x, false, w)) return;
    const int row0 = w.tile * S::RT, rows = min(S::RT, w.s.nq * u.g - row0), ctx = w.s.kv - w.s.nq;
    const int last = ctx + (row0 + rows - 1) / u.g;
    const int k_begin = w.split * w.chunk, k_end = min(last + 1, k_begin + w.chunk);
    if (k_begin >= k_end) return;

    uint8_t* ring = ring_sm + warp * S::STAGES * 2 * S::BLOCK;
    const float* pool = reinterpret_cast<const float*>(a.pool);
    const long long head_elems = (long long)HD << p.page_shift, v_off = p.Hkv * head_elems;
    const int n_groups = (k_end - k_begin + 15) / 16;
    const int mine = n_groups > warp ? (n_groups - warp + MMA_WARPS - 1) / MMA_WARPS : 0;
    auto key0 = [&](int i) { return k_begin + 16 * (warp + MMA_WARPS * i); };
    int pages = 0;
    auto copy = [&](int i) {
        if ((i & 31) == 0) pages = i + lane < mine ? max(load_page(p, w.b, key0(i + lane)), 0) : 0;
        const int page = __shfl_sync(0xffffffffu, pages, i & 31);
        if (lane == 0) {
            const float* src = pool + ((long long)page * 2 * p.Hkv + w.head) * head_elems +
                               (long long)(key0(i) & ((1 << p.page_shift) - 1)) * HD;
            uint8_t* dst = ring + i % S::STAGES * 2 * S::BLOCK;
            uint64_t* bar = &full[warp][i % S::STAGES];
            mbar_expect_tx(bar, 2 * S::BLOCK);
            bulk_load(dst, src, S::BLOCK, bar);
            bulk_load(dst + S::BLOCK, src + v_off, S::BLOCK, bar);
        }
    };
    for (int i = 0; i < S::STAGES && i < mine; ++i) copy(i);
    for (int i = threadIdx.x; i < S::RT * HD; i += MMA_WARPS * 32) {
        const int r = i / HD, row = row0 + r;
        float x = 0.f;
        if (r < rows)
            x = reinterpret_cast<const float*>(a.q)[(w.s.q0 + row / u.g) * a.q_stride +
                                                    (long long)(w.head * u.g + row % u.g) * HD + i % HD];
        qs[i] = x * (a.scale * LOG2E);
    }
    __syncthreads();

    float m[4], l[4], o[4][NC];                             // l: of this lane's keys
    int limit[4];                                           // the last key of rows 4 half + r
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = 4 * half + r;
        limit[r] = i < rows ? ctx + (row0 + i) / u.g : -1;
        m[r] = NEG_BIG;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) o[r][c] = 0.f;
    }
    bool ok = true;
    int done = 0;
    for (; done < mine; ++done) {
        ok = __all_sync(0xffffffffu, mbar_wait(&full[warp][done % S::STAGES], done / S::STAGES & 1, nullptr));
        if (!ok) break;
        const float* kb = reinterpret_cast<const float*>(ring + done % S::STAGES * 2 * S::BLOCK);
        const float* vb = kb + 16 * HD;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int c = 0; c < NP; ++c) {
            const int at = (c + k) % NP * 4;
            const float4 x = *reinterpret_cast<const float4*>(kb + k * HD + at);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float4 q = *reinterpret_cast<const float4*>(qs + (4 * half + r) * HD + at);
                s[r] = fmaf(q.x, x.x, fmaf(q.y, x.y, fmaf(q.z, x.z, fmaf(q.w, x.w, s[r]))));
            }
        }
        const int key = key0(done) + k;
        float mx[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (key > limit[r] || key >= k_end) s[r] = -INFINITY;
            mx[r] = fmaxf(m[r], s[r]);
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], d));
            const float al = ex2_approx(m[r] - mx[r]);
            m[r] = mx[r];
            s[r] = ex2_approx(s[r] - mx[r]);
            l[r] = l[r] * al + s[r];
#pragma unroll
            for (int c = 0; c < NC; ++c) o[r][c] *= al;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) ps[warp][4 * half + r][k] = s[r];
        __syncwarp();
        const int have = k_end - key0(done);                // (values behind the last key hold anything)
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            float4 pr[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) pr[r] = *reinterpret_cast<const float4*>(&ps[warp][4 * half + r][j]);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = j + e < have ? vb[(j + e) * HD + 16 * c + k] : 0.f;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    o[r][c] = fmaf(pr[r].x, v[0], fmaf(pr[r].y, v[1], fmaf(pr[r].z, v[2], fmaf(pr[r].w, v[3], o[r][c]))));
            }
        }
        __syncwarp();                                       // the stage is read
        if (done + S::STAGES < mine) copy(done + S::STAGES);
    }
    if (!ok && lane == 0) {
        raise_flag(p.hdr, ERR_TIMEOUT);
        // the copies in flight land before the shared memory is given back
        for (int i = done; i < mine && i < done + S::STAGES; ++i)
            mbar_wait(&full[warp][i % S::STAGES], i / S::STAGES & 1, nullptr);
    }
    if (__syncthreads_or(!ok)) return;                      // (behind it the rings are through)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
        float* dst = sm + (warp * S::RT + 4 * half + r) * S::LD;
#pragma unroll
        for (int c = 0; c < NC; ++c) dst[16 * c + k] = o[r][c];
        if (k == 0) { dst[HD] = m[r]; dst[HD + 1] = l[r]; }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * HD; i += MMA_WARPS * 32) {
        const int r = i / HD, col = i % HD;
        float mt = NEG_BIG;
#pragma unroll
        for (int x = 0; x < MMA_WARPS; ++x) mt = fmaxf(mt, sm[(x * S::RT + r) * S::LD + HD]);
        float lt = 0.f, acc = 0.f;
#pragma unroll
        for (int x = 0; x < MMA_WARPS; ++x) {
            const float* src = sm + (x * S::RT + r) * S::LD;
            const float f = ex2_approx(src[HD] - mt);
            lt += f * src[HD + 1];
            acc += f * src[col];
        }
        if (w.n_splits > 1) {
            float* pr = part_row(a, u, w.slot, r, HD);
            pr[col] = acc;
            if (col == 0) { pr[HD] = mt; pr[HD + 1] = lt; }
        } else {
            const int row = row0 + r;
            reinterpret_cast<float*>(a.o)[(long long)(w.s.q0 + row / u.g) * a.o_stride +
                                          (long long)(w.head * u.g + row % u.g) * HD + col] = acc / lt;
        }
    }
}

// Where the items alone would leave half the GPU idle they are cut into one unit for each of the
// `resident` CTAs (one sequence of 32000, 8 key heads of 128: 35 us, in nine pieces per SM 53 us), else
// into about nine per SM, so that ragged ones end together (32 contexts up to 16000: 185 us, in three per
// SM 216 us).  No unit is shorter than 256 keys, and where the items go round none is shorter than 1024,
// because joining costs a launch and the cut items' states.  (8 key heads of 128: 24 contexts up to 2000
// take 30 us with pieces of 256 and 34 us of 1024, 256 contexts up to 1000 take 139 us and 118 us.)  In
// float32 a key costs more and a row's join less beside it: few rows are cut until there is an item for
// every CTA (240 contexts and heads of 64 up to 2000: 48 us, in pieces of 1024 59 us; with tiles full of
// rows 50 us in place of 55 the other way round).
UnitPlan make_plan(const PagedArgs& p, int H, int rt, int rows_lo, int rows_hi, int resident) {
    UnitPlan u;
    u.g = H / p.Hkv;
    u.rt = rt;
    u.rows_lo = rows_lo;
    u.rows_hi = rows_hi;
    const long long items = plan_items(p, u);
    const bool idle = 2 * items < resident, few_rows = (long long)p.max_q * u.g <= F32Shape<16>::RT / 2;
    u.min_chunk = idle || (rt == F32Shape<16>::RT && few_rows && items < resident) ? 256 : 1024;
    u.chunk_align = 64;
    u.target = idle ? resident : 9 * sm_count();
    u.slots = (int)plan_slots(p, u);
    u.part = 0;
    return u;
}
constexpr int ANY = 1 << 30;
// CTAs per SM of the kernels for this head width (F32Shape, MmaShape)
template <template <int> class Shape>
int resident_ctas(int hd) {
    return sm_count() * (hd == 16 ? Shape<16>::CTAS : hd == 32 ? Shape<32>::CTAS : hd == 64 ? Shape<64>::CTAS : Shape<128>::CTAS);
}
UnitPlan f32_plan(const PagedArgs& p, int H, int hd) {
    return make_plan(p, H, F32Shape<16>::RT, 1, ANY, resident_ctas<F32Shape>(hd));
}

// bf16: sequences of at most FEW_ROWS rows per key head go to the warp-level kernel, those of more
// to the tcgen05 kernel, which head widths of 64 and 128 have (and pools whose rows TMA can count).
constexpr int FEW_ROWS = 16;
struct Bf16Plans {
    bool tc;
    UnitPlan u_mma;
    SharePlan u_tc;
    size_t floats;              // of partial states
};
Bf16Plans bf16_plans(const PagedArgs& p, int H, int hd) {
    Bf16Plans b;
    const int g = H / p.Hkv;
    b.tc = hd >= 64 && (long long)p.max_q * g > FEW_ROWS &&
           (((long long)p.n_pages * 2 * p.Hkv) << p.page_shift) < (1LL << 31);
    PagedArgs few = p;              // its bounds
    if (b.tc) few.max_q = FEW_ROWS / g < 1 ? 1 : FEW_ROWS / g;
    b.u_mma = make_plan(few, H, 16, 1, b.tc ? FEW_ROWS : ANY, resident_ctas<MmaShape>(hd));
    b.floats = (size_t)b.u_mma.slots * b.u_mma.rt * (hd + 2);
    b.u_tc = {};
    if (b.tc) {
        b.u_tc.g = g;
        b.u_tc.toks = 128 / g * PAGED_TC_STAGES;
        b.u_tc.rt = b.u_tc.toks * g;
        b.u_tc.rows_lo = FEW_ROWS + 1;
        b.u_tc.ctas = sm_count() * paged_tc_ctas(hd);
        // items of a few steps: cutting them would cost more than an uneven end
        b.u_tc.whole = p.max_kv <= 4 * STEP_KEYS;
        b.u_tc.part = (long long)b.floats;
        if (!b.u_tc.whole) {
            b.floats += (size_t)2 * b.u_tc.ctas * b.u_tc.rt * (hd + 2);
            b.floats = (b.floats + 3) / 4 * 4;
            b.u_tc.cuts = (long long)b.floats;
            b.floats += (size_t)b.u_tc.ctas * sizeof(ShareCut) / sizeof(float);
        }
    }
    return b;
}

template <int HD>
cudaError_t run_mma(Launch L, const PagedArgs& p, const PagedAttnArgs& a, const UnitPlan& u, long long items, bool beside_tc) {
    // A block per unit: blocks that walk through the units took 13 % longer for 64 decode contexts.  But
    // where another kernel has the long sequences there may be few units or none, and then blocks that
    // look for theirs in vain cost more: no more than are resident at once.
    const int units = (int)(items + (u.slots ? u.target : 0));
    const int most = sm_count() * MmaShape<HD>::CTAS, grid = beside_tc && units > most ? most : units;
    cudaError_t e = cudaFuncSetAttribute(k_paged_mma<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, MmaShape<HD>::SMEM);
    if (e != cudaSuccess) return e;
    return launch_k(L, k_paged_mma<HD>, (unsigned)grid, MMA_WARPS * 32, MmaShape<HD>::SMEM, p, a, u, units);
}

template <int HD>
cudaError_t run_f32(Launch L, const PagedArgs& p, const PagedAttnArgs& a, const UnitPlan& u) {
    cudaError_t e = cudaFuncSetAttribute(k_paged_f32<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, F32Shape<HD>::SMEM);
    if (e != cudaSuccess) return e;
    const long long grid = plan_items(p, u) + (u.slots ? u.target : 0);
    return launch_k(L, k_paged_f32<HD>, (unsigned)grid, MMA_WARPS * 32, F32Shape<HD>::SMEM, p, a, u);
}

// At most one cut item per two slots, `target` of them, and no more than there are items.
int join_items(const UnitPlan& u, long long items) {
    const long long n = items < u.target ? items : u.target;
    return u.slots == 0 ? 0 : (int)n;
}

// Blocks that share the rows of a cut item: as many as a tile can have rows, while the items alone do
// not fill the GPU.
int join_rows(const PagedArgs& p, const UnitPlan& u, int items) {
    const long long rows = (long long)p.max_q * u.g;
    const int most = rows < u.rt ? (int)rows : u.rt, want = (sm_count() * 8 + items - 1) / items;
    return want < most ? want : most;
}

}  // namespace

size_t paged_attn_workspace(const PagedArgs& p, int H, int hd, bool is_bf16) {
    if (!is_bf16) {
        const UnitPlan u = f32_plan(p, H, hd);
        return (size_t)u.slots * u.rt * (hd + 2) * sizeof(float);
    }
    return bf16_plans(p, H, hd).floats * sizeof(float);
}

template <>
cudaError_t launch_paged_attention<float>(Launch L, const PagedArgs& p, const PagedAttnArgs& a) {
    const UnitPlan u = f32_plan(p, a.H, a.hd);
    cudaError_t e = cudaErrorInvalidValue;
    switch (a.hd) {
        case 16: e = run_f32<16>(L, p, a, u); break;
        case 32: e = run_f32<32>(L, p, a, u); break;
        case 64: e = run_f32<64>(L, p, a, u); break;
        case 128: e = run_f32<128>(L, p, a, u); break;
    }
    const int n = join_items(u, plan_items(p, u));
    if (e != cudaSuccess || n == 0) return e;
    const int y = join_rows(p, u, n);
    return launch_k(L, k_paged_join<float>, dim3(n, y), JOIN_THREADS, 0, p, a, u, n, y, SharePlan{});
}
template <>
cudaError_t launch_paged_attention<bf16>(Launch L, const PagedArgs& p, const PagedAttnArgs& a) {
    const Bf16Plans b = bf16_plans(p, a.H, a.hd);
    // every sequence of few rows is one tile
    const long long mma_items = b.tc ? (long long)p.B * p.Hkv : plan_items(p, b.u_mma);
    cudaError_t e = cudaErrorInvalidValue;
    switch (a.hd) {
        case 16: e = run_mma<16>(L, p, a, b.u_mma, mma_items, b.tc); break;
        case 32: e = run_mma<32>(L, p, a, b.u_mma, mma_items, b.tc); break;
        case 64: e = run_mma<64>(L, p, a, b.u_mma, mma_items, b.tc); break;
        case 128: e = run_mma<128>(L, p, a, b.u_mma, mma_items, b.tc); break;
    }
    if (e == cudaSuccess && b.tc) e = launch_paged_tc(L, p, a, b.u_tc);
    if (e != cudaSuccess) return e;
    const int n1 = join_items(b.u_mma, mma_items), n2 = b.tc && !b.u_tc.whole ? b.u_tc.ctas - 1 : 0;
    if (n1 + n2 == 0) return e;
    const int y1 = n1 ? join_rows(p, b.u_mma, n1) : 1;
    const int y2 = n2 ? (b.u_tc.rt + JOIN_THREADS - 1) / JOIN_THREADS * (a.hd / JOIN_COLS) : 1;
    return launch_k(L, k_paged_join<bf16>, dim3(n1 + n2, y1 > y2 ? y1 : y2), JOIN_THREADS, 0, p, a, b.u_mma, n1, y1,
                    b.u_tc);
}

}  // namespace rlt
