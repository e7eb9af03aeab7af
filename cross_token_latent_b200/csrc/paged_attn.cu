// Causal attention of new tokens over a paged key/value cache: row r (token i of sequence b, at
// position t) reads keys 0 .. t of its sequence, query head j those of key head j / g.
//
// One pass over the keys with the running maximum and sum of the softmax.  Rows of one key head's
// group are taken together (rows are numbered i * g + j), so that shared keys are read once; a
// long key axis is cut into units (paged.cuh) whose partial states k_paged_join merges.
#include "paged.cuh"

namespace rlt {

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float NEG_BIG = -1e30f;

// Where a unit's results go: the output when its item is not cut, else a slot of partial states,
// per row head_dim accumulators (not divided by the sum), the maximum (of scaled base-2 scores)
// and the sum.
__device__ __forceinline__ float* part_row(const PagedAttnArgs& a, const UnitPlan& u, int slot, int row) {
    return a.part + ((long long)slot * u.rt + row) * (a.hd + 2);
}

// Joins the partial states of one cut item (block: one item, warps over its rows).
template <typename T>
__global__ void __launch_bounds__(128) k_paged_join(PagedArgs p, PagedAttnArgs a, UnitPlan u) {
    // The kernel in front waited for its predecessor before it let this one start, so the batch's
    // lengths may be read here; the partial states only behind the wait.
    Unit w;
    const bool any = find_unit(p, u, blockIdx.x, true, w);
    pdl_wait();
    pdl_trigger();
    if (!any) return;
    const int lane = threadIdx.x & 31, rows = w.s.nq * u.g;
    const int q = threadIdx.x >> 5;
    for (int i = q; i < u.rt; i += 4) {
        const int row = w.tile * u.rt + i;
        if (row >= rows) break;
        const int tok = row / u.g, keys = w.s.kv - w.s.nq + tok + 1;
        const int n = min(w.n_splits, (keys + w.chunk - 1) / w.chunk);     // units that saw a key of this row
        float m = NEG_BIG;
        for (int j = lane; j < n; j += 32) m = fmaxf(m, part_row(a, u, w.slot + j, i)[a.hd]);
        m = warp_max(m);
        float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
        for (int j = 0; j < n; ++j) {
            const float* r = part_row(a, u, w.slot + j, i);
            const float f = exp2f(r[a.hd] - m);
            l += f * r[a.hd + 1];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (c * 32 + lane < a.hd) acc[c] += f * r[c * 32 + lane];
        }
        const float inv = 1.0f / l;
        T* o = reinterpret_cast<T*>(a.o) + (w.s.q0 + tok) * a.o_stride + (long long)(w.head * u.g + row % u.g) * a.hd;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (c * 32 + lane < a.hd) o[c * 32 + lane] = from_f<T>(acc[c] * inv);
    }
}

// ------------------------------------------------------------------ CUDA cores
// 2 R rows of one key head against tiles of 64 keys in shared memory; thread t scores key t % 64
// for R rows, then owns a column of the output for some of the rows.  Float32 throughout.
template <typename T, int HD, int R>
__global__ void __launch_bounds__(128) k_paged_simt(PagedArgs p, PagedAttnArgs a, UnitPlan u) {
    constexpr int RT = 2 * R, KT = 64, LD = HD + 4;
    constexpr int GROUPS = 128 / HD, RPG = RT >= GROUPS ? RT / GROUPS : 1;      // rows per column group
    extern __shared__ __align__(16) float sm[];
    float* Ks = sm;                     // [KT][LD]
    float* Vs = Ks + KT * LD;           // [KT][HD]
    float* Qs = Vs + KT * HD;           // [RT][HD]
    float* Ps = Qs + RT * HD;           // [RT][KT]
    float* Al = Ps + RT * KT;           // [RT] rescale of the accumulators, then the sums
    pdl_wait();
    pdl_trigger();
    Unit w;
    if (!find_unit(p, u, blockIdx.x, false, w)) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rows = min(RT, w.s.nq * u.g - w.tile * RT);
    const int row0 = w.tile * RT, ctx = w.s.kv - w.s.nq;
    const int last = ctx + (row0 + rows - 1) / u.g;                 // the last key any row sees
    const int k_begin = w.split * w.chunk, k_end = min(last + 1, k_begin + w.chunk);
    if (k_begin >= k_end) return;                                   // this tile ends in front of the unit
    for (int i = tid; i < RT * HD; i += 128) {
        const int r = i / HD, row = row0 + r;
        float x = 0.f;
        if (r < rows)
            x = to_f(reinterpret_cast<const T*>(a.q)[(w.s.q0 + row / u.g) * a.q_stride +
                                                     (long long)(w.head * u.g + row % u.g) * HD + i % HD]);
        Qs[i] = x * (a.scale * LOG2E);
    }
    float m[RT / 4 > 0 ? RT / 4 : 1], l[RT / 4 > 0 ? RT / 4 : 1];   // of the rows this warp keeps
#pragma unroll
    for (int i = 0; i < (RT / 4 > 0 ? RT / 4 : 1); ++i) { m[i] = NEG_BIG; l[i] = 0.f; }
    float acc[RPG];
#pragma unroll
    for (int i = 0; i < RPG; ++i) acc[i] = 0.f;
    const int col = tid % HD, grp = tid / HD;
    constexpr int E = Vec16<T>::N, PIECES = HD / E;                 // 16-byte pieces of a key
    const T* pool = reinterpret_cast<const T*>(a.pool);
    const long long head_elems = (long long)HD << p.page_shift;
    for (int k0 = k_begin; k0 < k_end; k0 += KT) {
        __syncthreads();
        for (int i = tid; i < KT * PIECES; i += 128) {
            const int j = i / PIECES, c = (i % PIECES) * E, key = k0 + j;
            float kx[E], vx[E];
#pragma unroll
            for (int e = 0; e < E; ++e) kx[e] = vx[e] = 0.f;
            if (key < k_end) {
                const int page = max(load_page(p, w.b, key), 0);
                const long long at = ((long long)page * 2 * p.Hkv + w.head) * head_elems +
                                     (long long)(key & ((1 << p.page_shift) - 1)) * HD + c;
                Vec16<T>::unpack(ld16(pool + at), kx);
                Vec16<T>::unpack(ld16(pool + at + p.Hkv * head_elems), vx);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) { Ks[j * LD + c + e] = kx[e]; Vs[j * HD + c + e] = vx[e]; }
        }
        __syncthreads();
        {
            const int j = tid & 63, half = tid >> 6, key = k0 + j;
            float s[R];
#pragma unroll
            for (int r = 0; r < R; ++r) s[r] = 0.f;
            for (int c = 0; c < HD; c += 4) {
                const float4 k4 = *reinterpret_cast<const float4*>(&Ks[j * LD + c]);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float4 q4 = *reinterpret_cast<const float4*>(&Qs[(half * R + r) * HD + c]);
                    s[r] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, s[r]))));
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = half * R + r;
                const bool seen = row < rows && key < k_end && key <= ctx + (row0 + row) / u.g;
                Ps[row * KT + j] = seen ? s[r] : -INFINITY;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < (RT / 4 > 0 ? RT / 4 : 1); ++i) {
            const int r = warp + 4 * i;
            if (r < RT) {
                const float s0 = Ps[r * KT + lane], s1 = Ps[r * KT + lane + 32];
                const float mx = fmaxf(m[i], warp_max(fmaxf(s0, s1)));
                const float p0 = exp2f(s0 - mx), p1 = exp2f(s1 - mx), al = exp2f(m[i] - mx);
                l[i] = l[i] * al + warp_sum(p0 + p1);
                m[i] = mx;
                Ps[r * KT + lane] = p0;
                Ps[r * KT + lane + 32] = p1;
                if (lane == 0) Al[r] = al;
            }
        }
        __syncthreads();
        if (grp * RPG < RT) {
#pragma unroll
            for (int i = 0; i < RPG; ++i) acc[i] *= Al[grp * RPG + i];
            for (int j = 0; j < KT; j += 4) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = Vs[(j + e) * HD + col];
#pragma unroll
                for (int i = 0; i < RPG; ++i) {
                    const float4 p4 = *reinterpret_cast<const float4*>(&Ps[(grp * RPG + i) * KT + j]);
                    acc[i] = fmaf(p4.x, v[0], fmaf(p4.y, v[1], fmaf(p4.z, v[2], fmaf(p4.w, v[3], acc[i]))));
                }
            }
        }
    }
    __syncthreads();
    float* Mx = Ps;                     // the rows' maxima, beside their sums
#pragma unroll
    for (int i = 0; i < (RT / 4 > 0 ? RT / 4 : 1); ++i) {
        const int r = warp + 4 * i;
        if (r < RT && lane == 0) { Al[r] = l[i]; Mx[r] = m[i]; }
    }
    __syncthreads();
    if (grp * RPG < RT) {
#pragma unroll
        for (int i = 0; i < RPG; ++i) {
            const int r = grp * RPG + i, row = row0 + r;
            if (r < rows) {
                if (w.n_splits > 1) {
                    float* pr = part_row(a, u, w.slot, r);
                    pr[col] = acc[i];
                    if (col == 0) { pr[HD] = Mx[r]; pr[HD + 1] = Al[r]; }
                } else {
                    reinterpret_cast<T*>(a.o)[(w.s.q0 + row / u.g) * a.o_stride +
                                              (long long)(w.head * u.g + row % u.g) * HD + col] =
                        from_f<T>(acc[i] / Al[r]);
                }
            }
        }
    }
}

// Sequences of any number of rows; 2 rows per unit when no sequence has more, else 16.
UnitPlan simt_plan(const PagedArgs& p, int H) {
    UnitPlan u;
    u.g = H / p.Hkv;
    u.rt = (long long)p.max_q * u.g <= 2 ? 2 : 16;
    u.rows_lo = 1;
    u.rows_hi = 1 << 30;
    u.min_chunk = 256;
    u.chunk_align = 64;
    u.target = 148 * 8;
    u.slots = (int)plan_slots(p, u);
    return u;
}

template <typename T, int HD, int R>
cudaError_t run_simt(Launch L, const PagedArgs& p, const PagedAttnArgs& a, const UnitPlan& u) {
    constexpr int RT = 2 * R;
    constexpr size_t smem = (64 * (HD + 4) + 64 * HD + RT * HD + RT * 64 + RT) * sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(k_paged_simt<T, HD, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const long long grid = plan_items(p, u) + u.target;
    return launch_k(L, k_paged_simt<T, HD, R>, (unsigned)grid, 128, smem, p, a, u);
}
template <typename T, int R>
cudaError_t run_simt_hd(Launch L, const PagedArgs& p, const PagedAttnArgs& a, const UnitPlan& u) {
    switch (a.hd) {
        case 16: return run_simt<T, 16, R>(L, p, a, u);
        case 32: return run_simt<T, 32, R>(L, p, a, u);
        case 64: return run_simt<T, 64, R>(L, p, a, u);
        case 128: return run_simt<T, 128, R>(L, p, a, u);
    }
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t join(Launch L, const PagedArgs& p, const PagedAttnArgs& a, const UnitPlan& u) {
    if (u.slots == 0) return cudaSuccess;
    const long long items = plan_items(p, u);           // at most one cut item per two slots
    return launch_k(L, k_paged_join<T>, (unsigned)(items < u.target ? items : u.target), 128, 0, p, a, u);
}

}  // namespace

size_t paged_attn_workspace(const PagedArgs& p, int H, int hd, bool is_bf16) {
    const UnitPlan u = simt_plan(p, H);
    return (size_t)u.slots * u.rt * (hd + 2) * sizeof(float);
}

template <typename T>
cudaError_t launch_paged_attention(Launch L, const PagedArgs& p, const PagedAttnArgs& a) {
    const UnitPlan u = simt_plan(p, a.H);
    cudaError_t e = u.rt == 2 ? run_simt_hd<T, 1>(L, p, a, u) : run_simt_hd<T, 8>(L, p, a, u);
    return e == cudaSuccess ? join<T>(L, p, a, u) : e;
}
template cudaError_t launch_paged_attention<float>(Launch, const PagedArgs&, const PagedAttnArgs&);
template cudaError_t launch_paged_attention<bf16>(Launch, const PagedArgs&, const PagedAttnArgs&);

}  // namespace rlt
