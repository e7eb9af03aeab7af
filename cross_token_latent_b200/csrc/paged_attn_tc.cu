// Attention of many new rows over a paged cache on the sm_100a tensor cores (bf16, head_dim 64 or
// 128).  A CTA takes a tile of one key head's rows, two stages of up to 128 (rows of a group of
// query heads beside each other, so that shared keys are read once), against the keys of its unit
// in tiles of 128:
//   warp 8      TMA producer: the query tiles once, then K and V tiles alternately into a ring; a
//               tile is as many boxes as it has pages, one lane each
//   warp 9      TMEM allocation; the MMAs: S_s = Q_s K^T into the stage's 128 TMEM columns, then
//               O_s += P_s V with P_s read from TMEM and V as it lies in the page (MN-major)
//   warps 0-3   softmax of stage 0, warps 4-7 of stage 1, a thread per row: the scores leave TMEM
//               once, P_s goes back as bf16 over the scores' own columns.
// While one stage's rows are in the softmax the tensor core works on the other stage.  The
// running maximum moves only when it grew by more than 2^8 (RESCALE): a smaller maximum is as good
// a reference for the exponentials, and the accumulator then seldom has to be rescaled; a stage's
// O is final when its next scores have arrived, because the MMAs complete in order.
// Every mbarrier wait is bounded.
#include "paged.cuh"
#include "sm100.cuh"

namespace rlt {

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int KT = 128;                 // keys per tile
constexpr float RESCALE = 8.0f;         // log2: probabilities stay below 256

template <int HD>
struct TcShape {
    static constexpr int ATOMS = HD / 64;                   // 64-element swizzle atoms of a row
    static constexpr int Q_BYTES = 128 * HD * 2;            // one stage
    static constexpr int T_BYTES = KT * HD * 2;             // a tile of K or V
    static constexpr int SLOTS = HD == 128 ? 5 : 8;
    static constexpr int OFF_KV = 2 * Q_BYTES;
    static constexpr int OFF_BAR = OFF_KV + SLOTS * T_BYTES;
    static constexpr int SMEM = OFF_BAR + 256 + 1024;
    static constexpr uint32_t O_COL = 256;                  // S stages at 0 and 128, O stages behind
};
constexpr int TC_THREADS = 320;

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int HD>
__global__ void __launch_bounds__(TC_THREADS, 1)
k_paged_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmKV, PagedArgs p,
           PagedAttnArgs a, UnitPlan u, int q_box_bytes) {
    using S = TcShape<HD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);
    uint64_t* kv_full = q_full + 1;             // [SLOTS]
    uint64_t* kv_empty = kv_full + S::SLOTS;    // [SLOTS]
    uint64_t* s_full = kv_empty + S::SLOTS;     // [2] scores of tile j (phase j)
    uint64_t* p_full = s_full + 2;              // [2] probabilities of tile j, O rescaled
    uint64_t* o_done = p_full + 2;              // [2] the stage's last product
    uint64_t* drained = o_done + 2;             // after a timeout: the MMAs issued have completed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
    __shared__ int abort_flag;

    // No wait for the kernel in front here: it is the one that takes this batch's other sequences, it
    // lets this one start only behind its own wait for what came before, and neither reads what the
    // other writes.  The wait stands at the end, so that this kernel's completion covers that one's.
    Unit w;
    if (!find_unit(p, u, blockIdx.x, false, w)) {
        pdl_trigger();
        pdl_wait();
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = u.rt / 2;                  // rows per stage: whole tokens
    const int row0 = w.tile * u.rt, ctx = w.s.kv - w.s.nq;
    const int k_begin = w.split * w.chunk;
    int rows[2], nt[2];                         // of each stage: rows, key tiles
    int k_end = 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        rows[s] = max(0, min(half, w.s.nq * u.g - row0 - s * half));
        const int keys = rows[s] > 0 ? min(ctx + (row0 + s * half + rows[s] - 1) / u.g + 1, k_begin + w.chunk) : 0;
        nt[s] = max(0, (keys - k_begin + KT - 1) / KT);
        k_end = max(k_end, keys);
    }
    const int tiles = max(nt[0], nt[1]);
    if (tiles == 0) {
        pdl_trigger();
        pdl_wait();
        return;
    }

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        for (int s = 0; s < S::SLOTS; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 4);
            mbar_init(&o_done[s], 1);
        }
        mbar_init(drained, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // behind the allocation, which a kernel that starts early could otherwise get in front of
    pdl_trigger();

    if (warp == 8) {
        // lane i loads atom i % ATOMS of page i / ATOMS of a tile
        const int page_rows = min(KT, 1 << p.page_shift);
        const int pg = lane / S::ATOMS, atom = lane % S::ATOMS;
        if (lane == 0) mbar_expect_tx(q_full, (nt[0] > 0 ? q_box_bytes : 0) + (nt[1] > 0 ? q_box_bytes : 0));
        __syncwarp();
        if (lane < 2 * S::ATOMS && nt[pg] > 0)
            tma_load_3d(smem + pg * S::Q_BYTES + atom * 128 * 128, &tmQ, q_full, 64 * atom, w.head * u.g,
                        w.s.q0 + (row0 + pg * half) / u.g);
        bool ok = true;
        int done = 0;
        for (int j = 0; j < tiles && ok; ++j) {
            const int key = k_begin + j * KT + pg * page_rows;
            const bool mine = pg * page_rows < KT && key < k_end;
            const int boxes = min(KT / page_rows, (k_end - k_begin - j * KT + page_rows - 1) / page_rows) * S::ATOMS;
            const int page = mine ? max(load_page(p, w.b, key), 0) : 0;
            const int in_page = key & ((1 << p.page_shift) - 1);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const int item = 2 * j + kv, slot = item % S::SLOTS;
                ok = mbar_wait(&kv_empty[slot], ((item / S::SLOTS) & 1) ^ 1, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) mbar_expect_tx(&kv_full[slot], boxes * page_rows * 128);
                __syncwarp();
                if (mine)
                    tma_load_2d(smem + S::OFF_KV + slot * S::T_BYTES + atom * KT * 128 + pg * page_rows * 128, &tmKV,
                                &kv_full[slot], 64 * atom,
                                ((((page * 2 + kv) * p.Hkv + w.head) << p.page_shift)) + in_page);
                done = item + 1;
            }
        }
        if (!ok) {
            abort_flag = 1;
            // the copies in flight land before the shared memory is given back
            if (lane == 0) {
                mbar_wait(q_full, 0, nullptr);
                for (int i = max(0, done - S::SLOTS); i < done; ++i)
                    mbar_wait(&kv_full[i % S::SLOTS], (i / S::SLOTS) & 1, nullptr);
            }
        }
    } else if (warp == 9) {
        constexpr uint32_t id_s = idesc_bf16(128, KT), id_o = idesc_bf16(128, HD) | IDESC_B_MN;
        auto wait_kv = [&](int item) -> bool {
            const bool ok = mbar_wait(&kv_full[item % S::SLOTS], (item / S::SLOTS) & 1, &abort_flag);
            return __all_sync(0xffffffffu, ok);
        };
        auto issue_s = [&](int s, int j) {      // S_s = Q_s K_j^T
            if (lane == 0) {
                const uint8_t* kb = smem + S::OFF_KV + ((2 * j) % S::SLOTS) * S::T_BYTES;
#pragma unroll
                for (int at = 0; at < S::ATOMS; ++at) {
                    const uint64_t dq = sdesc_sw128(smem + s * S::Q_BYTES + at * 128 * 128);
                    const uint64_t dk = sdesc_sw128(kb + at * KT * 128);
#pragma unroll
                    for (int k = 0; k < 4; ++k) umma(tmem + s * 128, dq + 2 * k, dk + 2 * k, id_s, (at | k) != 0);
                }
                umma_commit(&s_full[s]);
            }
            __syncwarp();
        };
        bool ok = mbar_wait(q_full, 0, &abort_flag);
        ok = __all_sync(0xffffffffu, ok) && wait_kv(0);
        if (ok) {
            tc_fence_after();
            for (int s = 0; s < 2; ++s)
                if (nt[s] > 0) issue_s(s, 0);
            if (lane == 0) umma_commit(&kv_empty[0]);
            for (int j = 0; j < tiles; ++j) {
                const int item = 2 * j + 1, slot = item % S::SLOTS;
                uint8_t* vb = smem + S::OFF_KV + slot * S::T_BYTES;
                if (!(ok = wait_kv(item))) break;
                const int have = k_end - k_begin - j * KT;
                if (have < KT) {
                    // slots behind the last key hold anything, and 0 * NaN is NaN: they become zeros
                    for (int i = lane; i < (KT - have) * S::ATOMS * 8; i += 32) {
                        const int piece = i & 7, at = (i >> 3) % S::ATOMS, r = have + (i >> 3) / S::ATOMS;
                        *reinterpret_cast<uint4*>(vb + at * KT * 128 + r * 128 + piece * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (j + 1 < tiles && !(ok = wait_kv(item + 1))) break;
                for (int s = 0; s < 2; ++s) {
                    if (j >= nt[s]) continue;
                    ok = mbar_wait(&p_full[s], j & 1, &abort_flag);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    tc_fence_after();
                    if (lane == 0) {
                        const uint64_t dv = sdesc_mn_sw128(vb, KT * 128);
#pragma unroll
                        for (int k = 0; k < KT / 16; ++k)
                            umma_ta(tmem + S::O_COL + s * HD, tmem + s * 128 + k * 8, dv + k * (16 * 128 >> 4), id_o,
                                    (j | k) != 0);
                        if (j + 1 == nt[s]) umma_commit(&o_done[s]);
                    }
                    __syncwarp();
                    if (j + 1 < nt[s]) issue_s(s, j + 1);
                }
                if (!ok) break;
                if (lane == 0) {
                    umma_commit(&kv_empty[slot]);
                    if (j + 1 < tiles) umma_commit(&kv_empty[(item + 1) % S::SLOTS]);
                }
            }
        }
        if (!ok) {
            abort_flag = 1;
            if (lane == 0) {
                umma_commit(drained);
                mbar_wait(drained, 0, nullptr);
            }
        }
    } else {
        const int s = warp >> 2, r = (warp & 3) * 32 + lane;        // stage, row of the stage
        const uint32_t t_s = tmem + s * 128 + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t t_o = tmem + S::O_COL + s * HD + ((uint32_t)((warp & 3) * 32) << 16);
        const int row = row0 + s * half + r;
        const int limit = r < rows[s] ? ctx + row / u.g - k_begin : -1;     // last key, from the unit's first
        const float c2 = a.scale * LOG2E;
        float m = -INFINITY, l = 0.f;           // m of the scaled scores
        bool ok = true;
        for (int j = 0; j < nt[s]; ++j) {
            ok = mbar_wait(&s_full[s], j & 1, &abort_flag);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after();
            uint32_t x[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32_async(t_s + 32 * c, x[c]);
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_wait_ld(x[c]);
            const int seen = limit - j * KT;    // columns 0 .. seen of this tile are seen
            if (__any_sync(0xffffffffu, seen < KT - 1)) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (32 * c + i > seen) x[c][i] = 0xff800000u;       // -inf
            }
            float mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(x[c][i]));
            mx *= c2;
            // (a first maximum needs no rescale: the first product overwrites O, and l is 0)
            const bool grow = mx > m + RESCALE || m == -INFINITY;
            if (__any_sync(0xffffffffu, grow)) {
                const float to = grow ? mx : m;
                const float al = m == -INFINITY ? 1.f : ex2_approx(m - to);
                l *= al;
                m = to;
                if (j > 0) {
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
            const float neg = m == -INFINITY ? 0.f : -m;            // a row that has seen nothing yet
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float e0 = ex2_approx(fmaf(__uint_as_float(x[c][2 * i]), c2, neg));
                    const float e1 = ex2_approx(fmaf(__uint_as_float(x[c][2 * i + 1]), c2, neg));
                    __nv_bfloat162 h = __floats2bfloat162_rn(e0, e1);
                    pk[i] = *reinterpret_cast<uint32_t*>(&h);
                    l += e0 + e1;
                }
                tmem_st16_async(t_s + 16 * c, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[s]);
        }
        if (ok && nt[s] > 0) {
            ok = mbar_wait(&o_done[s], 0, &abort_flag);
            ok = __all_sync(0xffffffffu, ok);
        }
        if (!ok) {
            abort_flag = 1;
            if (lane == 0) raise_flag(p.hdr, ERR_TIMEOUT);
        } else if (nt[s] > 0) {
            tc_fence_after();
            const bool mine = r < rows[s];
            if (w.n_splits > 1) {
                float* pr = part_row(a, u, w.slot, s * half + r, HD);
#pragma unroll 1
                for (int c = 0; c < HD; c += 32) {
                    float ov[32];
                    tmem_ld32(t_o + c, ov);
                    if (mine) {
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            *reinterpret_cast<float2*>(pr + c + i) = make_float2(ov[i], ov[i + 1]);
                    }
                }
                if (mine) *reinterpret_cast<float2*>(pr + HD) = make_float2(m, l);
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
        }
    }
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

template <int HD>
cudaError_t run(Launch L, const PagedArgs& p, const PagedAttnArgs& a, const UnitPlan& u) {
    using S = TcShape<HD>;
    cudaError_t e = cudaFuncSetAttribute(k_paged_tc<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    const int toks = u.rt / 2 / u.g;            // tokens per stage
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
    const long long grid = plan_items(p, u) + (u.slots ? u.target : 0);
    return launch_k(L, k_paged_tc<HD>, (unsigned)grid, TC_THREADS, S::SMEM, tq, tkv, p, a, u, u.g * toks * 128 * S::ATOMS);
}

}  // namespace

cudaError_t launch_paged_tc(Launch L, const PagedArgs& p, const PagedAttnArgs& a, const UnitPlan& u) {
    return a.hd == 64 ? run<64>(L, p, a, u) : run<128>(L, p, a, u);
}

}  // namespace rlt
