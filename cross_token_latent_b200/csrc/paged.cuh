// What the kernels over a paged key/value cache share: the description of a ragged batch, its
// checks on the device, and the split of the attention's work into units.
//
// The pool is [n_pages][2][n_kv_heads][page_size][head_dim] (plane 0 keys, plane 1 values), so a
// page holds a contiguous [page_size][head_dim] block per head.  Token p of sequence b lies in
// page table[b * table_stride + p / page_size], slot p % page_size.
#pragma once

#include "kernels.cuh"

namespace rlt {

struct PagedArgs {
    int B, N, max_q, max_kv;
    const int32_t* q_start;     // [B + 1]
    const int32_t* kv_len;      // [B]
    const int32_t* table;       // [B, table_stride]
    long long table_stride;
    int page_shift;             // log2(page_size)
    int n_pages, Hkv;
    DevHeader* hdr;
};

// Rows q0 .. q0 + nq - 1 of the packed batch are the last nq of a sequence's kv tokens.
struct Seq {
    int q0, nq, kv;
};

// Sequence b's lengths.  Lengths that do not fit what the host was told (they would lead out of
// the page table, the packed rows or the rotary table) latch ERR_BAD_PAGE, and the sequence counts
// as one without new tokens.
__device__ __forceinline__ Seq load_seq(const PagedArgs& p, int b) {
    Seq s;
    s.q0 = p.q_start[b];
    const int q1 = p.q_start[b + 1];
    s.kv = p.kv_len[b];
    s.nq = 0;
    const bool rows_ok = s.q0 >= 0 && q1 >= s.q0 && q1 <= p.N && q1 - s.q0 <= p.max_q;
    const bool kv_ok = s.kv >= 0 && s.kv <= p.max_kv;
    if (rows_ok && kv_ok && s.kv >= q1 - s.q0)
        s.nq = q1 - s.q0;
    else
        raise_flag(p.hdr, ERR_BAD_PAGE);
    return s;
}

// The page that holds token t of sequence b (0 <= t < max_kv), or -1 (latched) if the table names
// none of the pool's.
__device__ __forceinline__ int load_page(const PagedArgs& p, int b, int t) {
    const int page = p.table[b * p.table_stride + (t >> p.page_shift)];
    if (page >= 0 && page < p.n_pages) return page;
    raise_flag(p.hdr, ERR_BAD_PAGE);
    return -1;
}

// The sequence that holds packed row r: the last b with q_start[b] <= r (empty sequences are
// skipped by that); its bounds are checked by load_seq.  -1 for a row in front of them all.
__device__ __forceinline__ int find_seq(const PagedArgs& p, int r) {
    int lo = -1, hi = p.B;              // q_start[lo] <= r < q_start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.q_start[mid] <= r) lo = mid; else hi = mid;
    }
    return lo;
}

// ------------------------------------------------------------------ units of attention work
// A sequence's rows (token i, query head j of a key head's group) are numbered i * g + j and cut
// into tiles of rt rows; an item is one tile of one key head.  An item reads the sequence's keys,
// and where they are more than `chunk`, the chunk's length in keys, it is cut into that many
// units, whose partial softmax states a second kernel joins.  chunk = max(min_chunk, all items'
// keys / target): about `target` units of equal length whatever the raggedness, at most
// target + items of them, and at most 2 target that belong to a cut item.
struct UnitPlan {
    int g;                      // query heads per key head
    int rt;                     // rows per tile
    int rows_lo, rows_hi;       // the kernel takes sequences of rows_lo <= nq * g <= rows_hi
    int min_chunk;              // a multiple of chunk_align
    int chunk_align;
    int target;
    int slots;                  // partial states that the workspace holds
    long long part;             // the first of them, in floats
};

struct Unit {
    int b;
    Seq s;
    int head, tile;
    int split, n_splits;        // this unit is keys [split * chunk, ...) of n_splits chunks
    int chunk;
    int slot;                   // of the unit's partial state (n_splits > 1)
};

__device__ __forceinline__ int seq_tiles(const UnitPlan& u, const Seq& s) {
    const int rows = s.nq * u.g;
    return rows >= u.rows_lo && rows <= u.rows_hi ? (rows + u.rt - 1) / u.rt : 0;
}

__device__ __forceinline__ int warp_iscan(int v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// Unit number `index` of the batch, found by a whole warp: false if there are fewer.  With
// cut_items the index counts cut items instead (for the kernel that joins their units).
__device__ __forceinline__ bool find_unit(const PagedArgs& p, const UnitPlan& u, int index, bool cut_items, Unit& out) {
    const int lane = threadIdx.x & 31;
    long long total = 0;
    Seq first = {0, 0, 0};              // of sequence `lane`, for the second look
    for (int b = lane; b < p.B; b += 32) {
        const Seq s = load_seq(p, b);
        if (b == lane) first = s;
        total += (long long)seq_tiles(u, s) * s.kv;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    total *= p.Hkv;
    long long c = (total + u.target - 1) / u.target;
    c = (c + u.chunk_align - 1) / u.chunk_align * u.chunk_align;
    const int chunk = c < u.min_chunk ? u.min_chunk : (c > (1 << 30) ? 1 << 30 : (int)c);
    int base = 0, slot_base = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        Seq s = first;
        if (b0 > 0) s = b0 + lane < p.B ? load_seq(p, b0 + lane) : Seq{0, 0, 0};
        const int tiles = seq_tiles(u, s) * p.Hkv;
        const int ns = s.kv > chunk ? (s.kv + chunk - 1) / chunk : 1;
        const int slots = ns > 1 ? tiles * ns : 0;
        const int mine = cut_items ? (ns > 1 ? tiles : 0) : tiles * ns;
        const int end = base + warp_iscan(mine, lane), slot_end = slot_base + warp_iscan(slots, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, index < end);
        if (hit) {
            const int src = __ffs(hit) - 1;
            out.b = b0 + src;
            out.s.q0 = __shfl_sync(0xffffffffu, s.q0, src);
            out.s.nq = __shfl_sync(0xffffffffu, s.nq, src);
            out.s.kv = __shfl_sync(0xffffffffu, s.kv, src);
            out.n_splits = __shfl_sync(0xffffffffu, ns, src);
            out.chunk = chunk;
            int i = index - __shfl_sync(0xffffffffu, end - mine, src);
            const bool counted = i >= 0;
            const int slot0 = __shfl_sync(0xffffffffu, slot_end - slots, src);
            // the last tiles of a sequence see the most keys: they start first
            if (cut_items) {
                out.split = 0;
            } else {
                out.split = i % out.n_splits;
                i /= out.n_splits;
            }
            out.head = i % p.Hkv;
            out.tile = seq_tiles(u, out.s) - 1 - i / p.Hkv;
            out.slot = slot0 + i * out.n_splits + out.split;
            // Starts that overlap count rows twice, so that there are more units than the host sized
            // for, even more than an int counts: those beyond are left out.
            if (counted && out.tile >= 0 && (out.n_splits == 1 || (out.slot >= 0 && out.slot < u.slots))) return true;
            raise_flag(p.hdr, ERR_BAD_PAGE);
            return false;
        }
        base = __shfl_sync(0xffffffffu, end, 31);
        slot_base = __shfl_sync(0xffffffffu, slot_end, 31);
    }
    return false;
}

// ------------------------------------------------------------------ shares of attention work
// The tcgen05 kernel takes its work as one long line of steps (a tile of rows against 128 keys):
// sequence by sequence, tile by tile, head by head, key by key, cut into equal shares, one per
// CTA.  A share begins and ends anywhere, so every CTA has the same work whatever the raggedness
// and the causal order; an item (a tile and head) is cut only where a share ends, which leaves at
// most two partial states per CTA.  A step counts the same whether its tile fills both of its stages of
// rows or one: alone, a stage waits for its own chain (9 turns with heads of 64, steps of one stage
// counted half: 122 us in place of 100).  With `whole` an item counts as one step and is never cut.
constexpr int STEP_KEYS = 128;
struct SharePlan {
    int g;                      // query heads per key head
    int rt, toks;               // rows and tokens per tile: rt = toks * g
    int rows_lo;                // the kernel takes sequences of at least that many rows
    int ctas;
    int whole;
    long long part;             // partial states, in floats: slots 2c and 2c + 1 are CTA c's
    long long cuts;             // a ShareCut per CTA behind them, in floats
};
// Where a share begins: the item, and how many of its steps belong to the shares in front.
struct ShareCut {
    Seq s;
    int tile, head, step;
    long long begin, share;     // the item's first step among all, steps per share
};

__device__ __forceinline__ int share_tiles(const SharePlan& u, const Seq& s) {
    return s.nq * u.g >= u.rows_lo ? (s.nq + u.toks - 1) / u.toks : 0;
}
// steps of one of the sequence's items: key tiles up to the last key that a row of the tile sees
__device__ __forceinline__ int share_keys(const SharePlan& u, const Seq& s, int tile) {
    return s.kv - s.nq + min(s.nq, (tile + 1) * u.toks);
}
__device__ __forceinline__ int share_steps(const SharePlan& u, const Seq& s, int tile) {
    return u.whole ? 1 : (share_keys(u, s, tile) + STEP_KEYS - 1) / STEP_KEYS;
}
// Sum over i < n of floor((a i + b) / m), reduced by the steps of Euclid's algorithm (sums of floors of an
// arithmetic progression: Graham, Knuth, Patashnik, Concrete Mathematics, 3.5).
__device__ __forceinline__ long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
    long long sum = 0;
    while (n > 0) {
        sum += (long long)n * (n - 1) / 2 * (a / m) + (long long)n * (b / m);
        a %= m;
        b %= m;
        const unsigned long long y = (unsigned long long)a * n + b;
        if (y < m) break;
        n = (unsigned)(y / m);
        b = (unsigned)(y % m);
        const unsigned t = m;
        m = a;
        a = t;
    }
    return sum;
}
// steps of all tiles of the sequence, for one head
__device__ __forceinline__ long long share_seq_steps(const SharePlan& u, const Seq& s) {
    const int tiles = share_tiles(u, s);
    if (tiles == 0 || u.whole) return tiles;
    const int full = s.nq / u.toks;
    long long n = floor_sum(full, STEP_KEYS, u.toks, s.kv - s.nq + u.toks + STEP_KEYS - 1);
    if (full < tiles) n += (s.kv + STEP_KEYS - 1) / STEP_KEYS;
    return n;
}

struct ShareStart {
    long long total, share;     // steps in all, per CTA
    int b;                      // the sequence that share number `index` begins in
    long long off;              // and the step within it (over its heads and tiles)
};
struct ShareSmem {
    long long warp[32];
    long long off;
    int b;
};
// Where share `index` begins; all threads of the block, false where there is no such share.
__device__ __forceinline__ bool find_share(const PagedArgs& p, const SharePlan& u, int index, ShareSmem& sm, ShareStart& out) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    long long mine = 0, first = 0;
    for (int b = tid; b < p.B; b += blockDim.x) {
        const long long n = share_seq_steps(u, load_seq(p, b)) * p.Hkv;
        if (b == tid) first = n;
        mine += n;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) sm.warp[warp] = mine;
    if (tid == 0) sm.b = -1;
    __syncthreads();
    long long total = 0;
    for (int i = 0; i < warps; ++i) total += sm.warp[i];
    // a share of a few steps at least: a CTA costs about two to set up
    const long long even = (total + u.ctas - 1) / u.ctas, least = u.whole ? 1 : 4;
    out.total = total;
    out.share = even > least ? even : least;
    const long long target = out.share * index;
    if (target >= total) return false;
    long long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += blockDim.x) {
        const int b = b0 + tid;
        const long long n = b0 == 0 ? first : (b < p.B ? share_seq_steps(u, load_seq(p, b)) * p.Hkv : 0);
        long long end = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += y;
        }
        __syncthreads();                    // sm.warp is free
        if (lane == 31) sm.warp[warp] = end;
        __syncthreads();
        long long before = base;
        for (int i = 0; i < warp; ++i) before += sm.warp[i];
        if (before + end - n <= target && target < before + end) {
            sm.b = b;
            sm.off = target - (before + end - n);
        }
        for (int i = 0; i < warps; ++i) base += sm.warp[i];
        __syncthreads();
        if (sm.b >= 0) break;
    }
    out.b = sm.b;
    out.off = sm.off;
    return out.b >= 0;
}
// The tile, head and step of step number off of a sequence, found by a whole warp.
__device__ __forceinline__ void locate_step(const SharePlan& u, const Seq& s, int Hkv, long long off, int& tile, int& head,
                                            int& step) {
    const int lane = threadIdx.x & 31, tiles = share_tiles(u, s);
    for (int t0 = 0; t0 < tiles; t0 += 32) {
        const int n = t0 + lane < tiles ? share_steps(u, s, t0 + lane) : 0;
        int end = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, off < (long long)end * Hkv);
        if (hit) {
            const int src = __ffs(hit) - 1, steps = __shfl_sync(0xffffffffu, n, src);
            const int rem = (int)(off - (long long)(__shfl_sync(0xffffffffu, end, src) - steps) * Hkv);
            tile = t0 + src;
            head = rem / steps;
            step = rem % steps;
            return;
        }
        off -= (long long)__shfl_sync(0xffffffffu, end, 31) * Hkv;
    }
    tile = head = step = 0;
}

// Bounds that the host knows: items of a plan, and the slots of its partial states.
inline long long plan_items(const PagedArgs& p, const UnitPlan& u) {
    const long long rows = (long long)p.N * u.g;
    const long long tiles = rows / u.rt + p.B;                      // sum of the rounded-up counts
    const long long most = (long long)p.B * (((long long)p.max_q * u.g + u.rt - 1) / u.rt);
    return (tiles < most ? tiles : most) * p.Hkv;
}
inline long long plan_slots(const PagedArgs& p, const UnitPlan& u) {
    if (p.max_kv <= u.min_chunk) return 0;
    const long long all = plan_items(p, u) * ((p.max_kv + u.min_chunk - 1) / u.min_chunk);
    return all < 2LL * u.target ? all : 2LL * u.target;
}

// ------------------------------------------------------------------ paged_append.cu
// Rows of k, v (and q) [N, heads, head_dim] with row strides in elements, in float32 or the
// storage type: rotated keys and the values into the pool, rotated queries into q_out.
struct AppendArgs {
    const void *k, *v, *q;
    long long k_stride, v_stride, q_stride, q_out_stride;
    void* q_out;
    int H;                      // query heads (0 without q)
    void* pool;
    const float2* rope;         // [max_pos][head_dim / 2]
    int hd;
};
template <typename T, typename S>
cudaError_t launch_paged_append(Launch L, const PagedArgs& p, const AppendArgs& a);
// Row r of ews [N, d] (token i of sequence b, position t) -> e[b, t], and of kv float32 [N, 2d] ->
// M_g [2][B][H][T_alloc][hd]
template <typename T>
cudaError_t launch_paged_scatter_e(Launch L, const PagedArgs& p, const T* ews, int d, T* e, int T_alloc);
template <typename T>
cudaError_t launch_paged_scatter_m(Launch L, const PagedArgs& p, const float* kv, int H, int hd, T* Mg, int T_alloc);

// ------------------------------------------------------------------ paged_attn.cu
struct PagedAttnArgs {
    const void* q;              // [N, H, hd], storage type
    void* o;                    // [N, H, hd], storage type
    long long q_stride, o_stride;   // elements between rows
    const void* pool;
    int H, hd;
    float scale;
    float* part;                // partial states of cut items
};
// A row of a cut item's partial state: head_dim accumulators (not divided by the sum), the maximum
// (of base-2 scaled scores) and the sum.
__device__ __forceinline__ float* part_row(const PagedAttnArgs& a, const UnitPlan& u, int slot, int row, int hd) {
    return a.part + u.part + ((long long)slot * u.rt + row) * (hd + 2);
}
// The partial state of a share plan's slot, [head_dim + 2][rt]: a thread has a row of it, and rows side
// by side make its accesses whole ones.
__device__ __forceinline__ float* share_part(const PagedAttnArgs& a, const SharePlan& u, int slot, int hd) {
    return a.part + u.part + (long long)slot * u.rt * (hd + 2);
}
size_t paged_attn_workspace(const PagedArgs& p, int H, int hd, bool is_bf16);
template <typename T>
cudaError_t launch_paged_attention(Launch L, const PagedArgs& p, const PagedAttnArgs& a);

// ------------------------------------------------------------------ paged_attn_tc.cu
constexpr int PAGED_TC_STAGES = 2;                                  // row stages of a tile
constexpr int paged_tc_ctas(int hd) { return hd == 64 ? 2 : 1; }    // CTAs per SM
cudaError_t launch_paged_tc(Launch L, const PagedArgs& p, const PagedAttnArgs& a, const SharePlan& u);

// ------------------------------------------------------------------ logits.cu
struct LogitsArgs {
    const float* x;             // [B, V], row stride x_stride
    long long x_stride;
    float* out;                 // may be x
    long long out_stride;
    int B, V;
    const float* lse;           // [B] or NULL
    const float* bias;          // [B, V] with row stride bias_stride (0: one row for all), or NULL
    long long bias_stride;
    const uint32_t* mask;       // [B, ceil(V / 32)] with row stride mask_stride (0: one row for all), or NULL
    long long mask_stride;
    const int32_t* tokens;      // history: token i of row b at tokens[b * seq_stride + i * tok_stride], or NULL
    long long seq_stride, tok_stride;
    int n_tokens;
    const int32_t* tok_len;     // [B] or NULL (n_tokens for every row)
    const int32_t* gen_start;   // [B] or NULL (0)
    const float *repetition, *presence, *frequency, *tau;       // [B] or NULL (1, 0, 0, 1)
    float* out_lse;             // [B] or NULL
    DevHeader* hdr;
};
int logits_max_vocab();
cudaError_t launch_process_logits(Launch L, const LogitsArgs& a);

}  // namespace rlt
