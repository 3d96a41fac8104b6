// kda_pages.cu -- pages of recurrent states (include/kda.h, kda_state_copy,
// kda_state_alloc, kda_state_free, kda_state_compact).  Copies are HBM-bound: 80
// pages of 2 MiB take 52 us, 6.4 TB/s of the 6.5 of one plain copy; 8 pages forked into
// 64 and 8 cleared 28 us (168 MB, 26 us at that rate).  The plans are one CTA: 4 us for 96
// pages, 14 us for 5,000.
#include "kda_launch.h"
#include "kda_sm100.cuh"

namespace kda {

namespace {

constexpr int COPY_THREADS = 256;
constexpr int COPY_UNROLL = 8;

struct CopyArgs {
    uint8_t* dst;
    const uint8_t* src;
    int64_t page_bytes, dst_layer, src_layer;
    int dst_pages, src_pages, n;
    bool same;  // dst and src are one pool
    const int32_t *dst_slots, *src_slots;
};

struct Entry {
    int d, s;   // s < 0: clear
    bool does;  // false: an entry that does nothing
};

KDA_DEV Entry entry(const CopyArgs& a, int i) {
    Entry e{a.dst_slots[i], a.src_slots[i], true};
    if (e.s < 0) e.s = -1;
    e.does = e.d >= 0 && e.d < a.dst_pages && e.s < a.src_pages && !(a.same && e.s == e.d);
    return e;
}

// One CTA = one piece (COPY_THREADS x COPY_UNROLL vectors) of the pages of one entry of the list, or of every 1,024th of
// a long one, in one layer.  The list's order only matters where an entry reads or writes a page that another one writes
// ("tied" entries).  All others are copied side by side.  The tied ones are carried out one after the other by the
// CTAs of the first of them: a thread moves the same bytes of every page, so its own program order is the list's order.
// Which entries are tied is looked up in three sets of pages (written, written twice, read) that each CTA makes in one pass
// over the list; a set has a bit per page, or per page modulo 131,072 in larger pools, where a page may be taken for
// another: an entry that is tied by mistake gets the same result, a little later.  1,000 pages of 512 KB: 191 us, 5.5 TB/s,
// with half of them in one chain 441 us; 30,000 of 256 bytes 119 us (1.2 ms where each entry looked through the list
// for itself, and the first tied one for all others); 64 pages of 2 MiB 43 us, 64 in one chain 41 us.
constexpr int COPY_ENTRIES = 1024;
constexpr int COPY_MAX_BITS = 131072;  // three sets: the 48 KB of shared memory that a CTA has without asking

template <typename V>
__global__ void __launch_bounds__(COPY_THREADS) state_copy_kernel(CopyArgs a, int words) {
    extern __shared__ uint32_t sets[];
    uint32_t *const written = sets, *const twice = sets + words, *const read = sets + 2 * words;
    const int tid = threadIdx.x, mask = 32 * words - 1;
    bool any = false;
    for (int i = blockIdx.y; i < a.n; i += gridDim.y) any |= entry(a, i).does;
    if (!any) return;
    for (int w = tid; w < 3 * words; w += COPY_THREADS) sets[w] = 0;
    __syncthreads();
    for (int j = tid; j < a.n; j += COPY_THREADS) {
        const Entry o = entry(a, j);
        if (!o.does) continue;
        const int d = o.d & mask, s = o.s & mask;
        if (atomicOr(&written[d >> 5], 1u << (d & 31)) >> (d & 31) & 1) atomicOr(&twice[d >> 5], 1u << (d & 31));
        if (a.same && o.s >= 0) atomicOr(&read[s >> 5], 1u << (s & 31));
    }
    __syncthreads();
    auto has = [&](const uint32_t* set, int page) { return (set[(page & mask) >> 5] >> (page & 31) & 1) != 0; };
    auto tied = [&](const Entry& e) {
        return e.does && (has(twice, e.d) || (a.same && (has(read, e.d) || (e.s >= 0 && has(written, e.s)))));
    };

    uint8_t* const dst = a.dst + (int64_t)blockIdx.z * a.dst_layer;
    const uint8_t* const src = a.src + (int64_t)blockIdx.z * a.src_layer;
    const int64_t n_vec = a.page_bytes / (int64_t)sizeof(V);
    const int64_t v0 = (int64_t)blockIdx.x * (COPY_THREADS * COPY_UNROLL) + tid;
    auto move = [&](const Entry& ek) {
        V* const to = reinterpret_cast<V*>(dst + (int64_t)ek.d * a.page_bytes);
        const V* const from = reinterpret_cast<const V*>(src + (int64_t)(ek.s < 0 ? 0 : ek.s) * a.page_bytes);
        V v[COPY_UNROLL];
#pragma unroll
        for (int u = 0; u < COPY_UNROLL; ++u) {
            const int64_t at = v0 + (int64_t)u * COPY_THREADS;
            v[u] = V{};
            if (ek.s >= 0 && at < n_vec) v[u] = from[at];
        }
#pragma unroll
        for (int u = 0; u < COPY_UNROLL; ++u) {
            const int64_t at = v0 + (int64_t)u * COPY_THREADS;
            if (at < n_vec) to[at] = v[u];
        }
    };

    int first_mine = a.n;  // the first tied entry of this CTA's
    for (int i = blockIdx.y; i < a.n; i += gridDim.y) {
        const Entry e = entry(a, i);
        if (!tied(e)) {
            if (e.does) move(e);
        } else if (first_mine == a.n) {
            first_mine = i;
        }
    }
    bool earlier = first_mine == a.n;
    for (int k = tid; k < first_mine && !earlier; k += COPY_THREADS) earlier = tied(entry(a, k));
    if (__syncthreads_or(earlier)) return;
    for (int k0 = first_mine; k0 < a.n; k0 += 32) {  // every warp for itself
        const int k = k0 + (tid & 31);
        for (unsigned left = __ballot_sync(0xffffffffu, k < a.n && tied(entry(a, k))); left; left &= left - 1)
            move(entry(a, k0 + __ffs(left) - 1));
    }
}

// The plans: one CTA of 1024 threads.
constexpr int PLAN_THREADS = 1024;

// Number of set flags before this thread's within the CTA, and their total.
KDA_DEV int block_rank(bool flag, int* total) {
    __shared__ int s_warp[PLAN_THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned m = __ballot_sync(0xffffffffu, flag);
    __syncthreads();  // the last call's values have been read
    if (lane == 0) s_warp[warp] = __popc(m);
    __syncthreads();
    int before = __popc(m & ((1u << lane) - 1u)), sum = 0;
    for (int k = 0; k < PLAN_THREADS / 32; ++k) {
        if (k < warp) before += s_warp[k];
        sum += s_warp[k];
    }
    *total = sum;
    return before;
}

__global__ void __launch_bounds__(PLAN_THREADS)
state_compact_kernel(uint8_t* live, int P, int32_t* dst_slots, int32_t* src_slots, int32_t* new_slots,
                     int32_t* n_live) {
    int m = 0;
    for (int p0 = 0; p0 < P; p0 += PLAN_THREADS) {
        const int p = p0 + threadIdx.x;
        int total;
        block_rank(p < P && live[p], &total);
        m += total;
    }
    int holes = 0, tails = 0;  // so far
    for (int p0 = 0; p0 < P; p0 += PLAN_THREADS) {
        const int p = p0 + threadIdx.x;
        const bool in = p < P, lv = in && live[p];
        int total;
        const int hk = holes + block_rank(in && !lv && p < m, &total);
        holes += total;
        const int tk = tails + block_rank(lv && p >= m, &total);
        tails += total;
        if (in && !lv && p < m) dst_slots[hk] = p;
        if (lv && p >= m) src_slots[tk] = p;
        if (in) new_slots[p] = lv && p < m ? p : -1;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < holes; k += PLAN_THREADS) new_slots[src_slots[k]] = dst_slots[k];
    for (int k = holes + threadIdx.x; k < P; k += PLAN_THREADS) dst_slots[k] = src_slots[k] = -1;
    for (int p = threadIdx.x; p < P; p += PLAN_THREADS) live[p] = p < m;
    if (threadIdx.x == 0) *n_live = m;
}

__global__ void __launch_bounds__(PLAN_THREADS) state_alloc_kernel(uint8_t* live, int P, int32_t* slots, int n) {
    int found = 0;
    for (int p0 = 0; p0 < P && found < n; p0 += PLAN_THREADS) {
        const int p = p0 + threadIdx.x;
        const bool is_free = p < P && !live[p];
        int total;
        const int k = found + block_rank(is_free, &total);
        if (is_free && k < n) {
            slots[k] = p;
            live[p] = 1;
        }
        found += total;
    }
    for (int k = found + threadIdx.x; k < n; k += PLAN_THREADS) slots[k] = -1;
}

__global__ void __launch_bounds__(256) state_free_kernel(uint8_t* live, int P, const int32_t* slots, int n) {
    const unsigned i = blockIdx.x * 256u + threadIdx.x;  // beyond 2^31 in the last CTA of the longest lists
    if (i >= (unsigned)n) return;
    const int s = slots[i];
    if (s >= 0 && s < P) live[s] = 0;
}

}  // namespace

cudaError_t launch_state_copy(void* dst, const void* src, int layers, int64_t page_bytes, int dst_pages, int src_pages,
                              int64_t dst_layer, int64_t src_layer, const int32_t* dst_slots,
                              const int32_t* src_slots, int n, cudaStream_t stream) {
    CopyArgs a{(uint8_t*)dst, (const uint8_t*)src, page_bytes, dst_layer, src_layer, dst_pages,
               src_pages, n, dst == src, dst_slots, src_slots};
    const bool wide = page_bytes % 16 == 0 && dst_layer % 16 == 0 && src_layer % 16 == 0;
    const int64_t n_vec = page_bytes / (wide ? 16 : 4);
    const int64_t per = COPY_THREADS * COPY_UNROLL;
    const dim3 grid((unsigned)((n_vec + per - 1) / per), (unsigned)(n < COPY_ENTRIES ? n : COPY_ENTRIES), (unsigned)layers);
    const int pages = a.same && src_pages > dst_pages ? src_pages : dst_pages;
    int words = 1;
    while (32 * words < pages && 32 * words < COPY_MAX_BITS) words *= 2;
    const size_t smem = 3 * words * sizeof(uint32_t);
    if (wide) state_copy_kernel<uint4><<<grid, COPY_THREADS, smem, stream>>>(a, words);
    else state_copy_kernel<uint32_t><<<grid, COPY_THREADS, smem, stream>>>(a, words);
    return cudaGetLastError();
}

cudaError_t launch_state_compact(uint8_t* live, int P, int32_t* dst_slots, int32_t* src_slots, int32_t* new_slots,
                                 int32_t* n_live, cudaStream_t stream) {
    state_compact_kernel<<<1, PLAN_THREADS, 0, stream>>>(live, P, dst_slots, src_slots, new_slots, n_live);
    return cudaGetLastError();
}

cudaError_t launch_state_alloc(uint8_t* live, int P, int32_t* slots, int n, cudaStream_t stream) {
    state_alloc_kernel<<<1, PLAN_THREADS, 0, stream>>>(live, P, slots, n);
    return cudaGetLastError();
}

cudaError_t launch_state_free(uint8_t* live, int P, const int32_t* slots, int n, cudaStream_t stream) {
    state_free_kernel<<<((unsigned)n + 255u) / 256u, 256, 0, stream>>>(live, P, slots, n);
    return cudaGetLastError();
}

}  // namespace kda
