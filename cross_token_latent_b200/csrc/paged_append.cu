// Append of new tokens to a paged key/value cache, the rotation by the token's position applied
// on the way, and the scatter of packed rows to a batch's encoder outputs.
//
// The append moves N (H + 2 Hkv) head_dim elements in and as many out and does three operations
// per rotated element: memory bounds it.  One launch takes queries, keys and values, so that the
// packed projection is read once and each row's sequence, position and angles are looked up once
// per warp's share of it.
#include "paged.cuh"

namespace rlt {

namespace {

// V consecutive elements as floats.
template <int V>
__device__ __forceinline__ void load_vec(const float* p, float* x) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const float4 q = *reinterpret_cast<const float4*>(p + i);
        x[i] = q.x; x[i + 1] = q.y; x[i + 2] = q.z; x[i + 3] = q.w;
    }
}
template <int V>
__device__ __forceinline__ void load_vec(const bf16* p, float* x) {
    if (V == 8) {
        Vec16<bf16>::unpack(ld16(p), x);
    } else {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        x[0] = __uint_as_float(w.x << 16); x[1] = __uint_as_float(w.x & 0xffff0000u);
        x[2] = __uint_as_float(w.y << 16); x[3] = __uint_as_float(w.y & 0xffff0000u);
    }
}
template <int V>
__device__ __forceinline__ void store_vec(float* p, const float* x) {
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}
template <int V>
__device__ __forceinline__ void store_vec(bf16* p, const float* x) {
    if (V == 8) {
        st16(p, Vec16<bf16>::pack(x));
    } else {
        __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
    }
}

// A work item is VEC elements f .. of a head's lower half together with their partners in the
// upper half; the items of a row are its query heads', its key heads', its value heads'.  A thread
// has the same item of every row it walks through, so that only the row's place is to be looked up,
// and its elements of the next row are on their way meanwhile: where they come from depends on the
// row's number alone.
template <typename T, typename S, int VEC>
__global__ void __launch_bounds__(256) k_paged_append(PagedArgs p, AppendArgs a) {
    pdl_wait();
    pdl_trigger();
    const int half = a.hd / 2, per_head = half / VEC;
    const int i = blockIdx.y * blockDim.x + threadIdx.x;
    if (i >= (a.H + 2 * p.Hkv) * per_head) return;
    const int head = i / per_head, f = (i % per_head) * VEC, h = head - a.H;
    const bool is_q = head < a.H, is_v = h >= p.Hkv;
    const int hk = is_v ? h - p.Hkv : h;
    const long long stride = is_q ? a.q_stride : (is_v ? a.v_stride : a.k_stride);
    const S* src = reinterpret_cast<const S*>(is_q ? a.q : (is_v ? a.v : a.k)) + (long long)(is_q ? head : hk) * a.hd + f;
    T* const dst_q = reinterpret_cast<T*>(a.q_out) + (long long)head * a.hd + f;
    T* const dst_kv = reinterpret_cast<T*>(a.pool) + f;
    float lo[VEC], hi[VEC];
    int r = blockIdx.x;
    load_vec<VEC>(src + r * stride, lo);
    load_vec<VEC>(src + r * stride + half, hi);
    for (; r < p.N; r += gridDim.x) {
        float next_lo[VEC], next_hi[VEC];
        const int rn = r + gridDim.x;
        if (rn < p.N) {
            load_vec<VEC>(src + rn * stride, next_lo);
            load_vec<VEC>(src + rn * stride + half, next_hi);
        }
        const int b = find_seq(p, r);
        Seq s = {0, 0, 0};
        if (b >= 0) s = load_seq(p, b);
        if (r < s.q0 + s.nq) {                          // no row behind the last sequence
            const int pos = s.kv - s.nq + (r - s.q0);
            T* dst = dst_q + r * a.q_out_stride;
            bool ok = true;
            if (!is_q) {
                const int page = load_page(p, b, pos), slot = pos & ((1 << p.page_shift) - 1);
                ok = page >= 0;
                dst = dst_kv + (((((long long)page * 2 + is_v) * p.Hkv + hk) << p.page_shift) + slot) * a.hd;
            }
            if (!is_v) {
                const float4* cs = reinterpret_cast<const float4*>(a.rope + (long long)pos * half + f);
#pragma unroll
                for (int j = 0; j < VEC; j += 2) {
                    const float4 t = __ldg(cs + j / 2);
                    const float x0 = lo[j], y0 = hi[j], x1 = lo[j + 1], y1 = hi[j + 1];
                    lo[j] = x0 * t.x - y0 * t.y;
                    hi[j] = x0 * t.y + y0 * t.x;
                    lo[j + 1] = x1 * t.z - y1 * t.w;
                    hi[j + 1] = x1 * t.w + y1 * t.z;
                }
            }
            if (ok) {
                store_vec<VEC>(dst, lo);
                store_vec<VEC>(dst + half, hi);
            }
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            lo[j] = next_lo[j];
            hi[j] = next_hi[j];
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(128) k_paged_scatter_e(PagedArgs p, const T* __restrict__ ews, int d,
                                                         T* __restrict__ e, int T_alloc) {
    pdl_wait();
    pdl_trigger();
    constexpr int N16 = Vec16<T>::N;
    for (int r = blockIdx.x; r < p.N; r += gridDim.x) {
        const int b = find_seq(p, r);
        if (b < 0) continue;
        const Seq s = load_seq(p, b);
        if (r >= s.q0 + s.nq) continue;
        const long long pos = s.kv - s.nq + (r - s.q0);
        for (int c = threadIdx.x * N16; c < d; c += blockDim.x * N16)      // d is a multiple of 8
            st16(e + ((long long)b * T_alloc + pos) * d + c, ld16(ews + (long long)r * d + c));
    }
}

template <typename T>
__global__ void __launch_bounds__(128) k_paged_scatter_m(PagedArgs p, const float* __restrict__ kv, int H, int hd,
                                                         T* __restrict__ Mg, int T_alloc) {
    pdl_wait();
    pdl_trigger();
    const int d = H * hd;
    const long long plane = (long long)p.B * H * T_alloc * hd;
    for (int r = blockIdx.x; r < p.N; r += gridDim.x) {
        const int b = find_seq(p, r);
        if (b < 0) continue;
        const Seq s = load_seq(p, b);
        if (r >= s.q0 + s.nq) continue;
        const long long pos = s.kv - s.nq + (r - s.q0);
        for (int c = threadIdx.x * 4; c < 2 * d; c += blockDim.x * 4) {
            float x[4];
            load_vec<4>(kv + (long long)r * 2 * d + c, x);
            const int sel = c >= d, h = (c - sel * d) / hd, f = (c - sel * d) % hd;
            store_vec<4>(Mg + sel * plane + (((long long)b * H + h) * T_alloc + pos) * hd + f, x);
        }
    }
}

inline unsigned rows_grid(long long n) {
    const long long most = 8LL * sm_count();
    return (unsigned)(n < most ? n : most);
}

}  // namespace

// Threads per SM that walk through the rows (32768 rows, heads of 128: 2048 take 223 us, 4096 take 201 us).
constexpr int ROW_THREADS = 4096;

template <typename T, typename S>
cudaError_t launch_paged_append(Launch L, const PagedArgs& p, const AppendArgs& a) {
    // 16 bytes per load: 4 float32 elements, 8 in bf16 (heads of 16 have halves of 8)
    constexpr int VEC = 16 / sizeof(S);
    // Rows of few items have small blocks (42000 float32 rows of 40 items: 44 us in blocks of 256, 32 us in blocks of 64).
    const int items = (a.H + 2 * p.Hkv) * (a.hd / (2 * VEC)), chunks = (items + 255) / 256;
    const int threads = ((items + chunks - 1) / chunks + 31) / 32 * 32;
    const int most = (ROW_THREADS * sm_count() + chunks * threads - 1) / (chunks * threads);
    return launch_k(L, k_paged_append<T, S, VEC>, dim3(p.N < most ? p.N : most, chunks), threads, 0, p, a);
}

template <typename T>
cudaError_t launch_paged_scatter_e(Launch L, const PagedArgs& p, const T* ews, int d, T* e, int T_alloc) {
    return launch_k(L, k_paged_scatter_e<T>, rows_grid(p.N), 128, 0, p, ews, d, e, T_alloc);
}
template <typename T>
cudaError_t launch_paged_scatter_m(Launch L, const PagedArgs& p, const float* kv, int H, int hd, T* Mg, int T_alloc) {
    return launch_k(L, k_paged_scatter_m<T>, rows_grid(p.N), 128, 0, p, kv, H, hd, Mg, T_alloc);
}

template cudaError_t launch_paged_append<float, float>(Launch, const PagedArgs&, const AppendArgs&);
template cudaError_t launch_paged_append<bf16, float>(Launch, const PagedArgs&, const AppendArgs&);
template cudaError_t launch_paged_append<bf16, bf16>(Launch, const PagedArgs&, const AppendArgs&);
template cudaError_t launch_paged_scatter_e<float>(Launch, const PagedArgs&, const float*, int, float*, int);
template cudaError_t launch_paged_scatter_e<bf16>(Launch, const PagedArgs&, const bf16*, int, bf16*, int);
template cudaError_t launch_paged_scatter_m<float>(Launch, const PagedArgs&, const float*, int, int, float*, int);
template cudaError_t launch_paged_scatter_m<bf16>(Launch, const PagedArgs&, const float*, int, int, bf16*, int);

}  // namespace rlt
