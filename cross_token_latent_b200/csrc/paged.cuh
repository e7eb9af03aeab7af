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
    for (int b = lane; b < p.B; b += 32) {
        const Seq s = load_seq(p, b);
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
        Seq s = {0, 0, 0};
        if (b0 + lane < p.B) s = load_seq(p, b0 + lane);
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
            // for: those beyond are left out.
            if (out.tile >= 0 && out.slot >= 0 && (out.n_splits == 1 || out.slot < u.slots)) return true;
            raise_flag(p.hdr, ERR_BAD_PAGE);
            return false;
        }
        base = __shfl_sync(0xffffffffu, end, 31);
        slot_base = __shfl_sync(0xffffffffu, slot_end, 31);
    }
    return false;
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
size_t paged_attn_workspace(const PagedArgs& p, int H, int hd, bool is_bf16);
template <typename T>
cudaError_t launch_paged_attention(Launch L, const PagedArgs& p, const PagedAttnArgs& a);

// ------------------------------------------------------------------ paged_attn_tc.cu
cudaError_t launch_paged_tc(Launch L, const PagedArgs& p, const PagedAttnArgs& a, const UnitPlan& u);

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
