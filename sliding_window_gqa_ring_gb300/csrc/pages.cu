// pages.cu -- copying, forking and moving the pages of a shared pool on the device.
//
// Every operator is a list of jobs "rows [0, n) of page s into page d", for keys, values
// and (e4m3 pages) the scales of the blocks those rows lie in, plus the page tables that
// name the pages.  Sources and destinations are lists in device memory, so a captured
// step follows what earlier kernels decided.
//
// Bytes: each copied byte is read once and written once; nothing else bounds a large
// call.  A CTA copies one piece of kPieceBytes of the keys or the values of one job, each
// thread kInFlight vectors of 16 bytes, all loaded before the first is stored.
#include "carat_internal.cuh"

namespace carat {
namespace {

constexpr int kCopyThreads = 256, kInFlight = 8;
constexpr long long kPieceBytes = (long long)kCopyThreads * kInFlight * 16;
constexpr int kMapSources = 1024;   // sources of a move kept in shared memory at a time

__device__ __forceinline__ bool page_ok(const PagesParams &p, int page) {
    return page >= 0 && page < p.num_pages;
}

// This CTA's piece of a job (blockIdx.x: pieces of the keys, then of the values, then one
// CTA for the scales).
__device__ void copy_piece(const PagesParams &p, int src, int dst, int rows) {
    if (src == dst || rows == 0) return;
    const int piece = blockIdx.x;
    if (piece < 2 * p.pieces) {
        char *base = static_cast<char *>(piece < p.pieces ? p.key_pages : p.value_pages);
        if (!base) return;
        const long long first = (long long)(piece % p.pieces) * kPieceBytes;
        const long long vectors = (rows * p.row_bytes - first) / 16;
        if (vectors <= 0) return;
        const long long page_bytes = p.page_rows * p.row_bytes;
        const uint4 *from = reinterpret_cast<const uint4 *>(base + src * page_bytes + first);
        uint4 *to = reinterpret_cast<uint4 *>(base + dst * page_bytes + first);
        uint4 v[kInFlight];
#pragma unroll
        for (int i = 0; i < kInFlight; ++i)
            if (i * kCopyThreads + (int)threadIdx.x < vectors)
                v[i] = __ldcs(from + i * kCopyThreads + threadIdx.x);
#pragma unroll
        for (int i = 0; i < kInFlight; ++i)
            if (i * kCopyThreads + (int)threadIdx.x < vectors)
                __stcs(to + i * kCopyThreads + threadIdx.x, v[i]);
        return;
    }
    if (!p.k_scales) return;
    const int page_words = p.page_rows / p.block_rows * p.kv_heads;
    const int words = (rows + p.block_rows - 1) / p.block_rows * p.kv_heads;
    for (int i = threadIdx.x; i < words; i += kCopyThreads) {
        p.k_scales[(long long)dst * page_words + i] = p.k_scales[(long long)src * page_words + i];
        p.v_scales[(long long)dst * page_words + i] = p.v_scales[(long long)src * page_words + i];
    }
}

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const PagesParams p) {
    wait_for_prior_launch();
    let_next_launch_start();
    for (int job = blockIdx.y; job < p.count; job += gridDim.y) {
        const int src = p.src[job], dst = p.dst[job];
        if (src < 0) continue;
        const int rows = p.rows ? p.rows[job] : p.page_rows;
        int bad = page_ok(p, src) && page_ok(p, dst) ? 0 : CARAT_DEV_BAD_CACHE_ID;
        if (rows < 0 || rows > p.page_rows) bad |= CARAT_DEV_BAD_CONTEXT;
        if (bad) {
            if (blockIdx.x == 0 && threadIdx.x == 0) set_status(p.dev_status, bad);
            continue;
        }
        copy_piece(p, src, dst, rows);
    }
}

// Child job of parent q: whole pages by name, the partial page by its rows.  blockIdx.x =
// 2 * pieces + 1 writes the child's line of the table and its length.
__global__ void __launch_bounds__(kCopyThreads) paged_fork_kernel(const PagesParams p) {
    wait_for_prior_launch();
    let_next_launch_start();
    for (int job = blockIdx.y; job < p.count; job += gridDim.y) {
        const int parent = p.parents[job];
        if (parent < 0) continue;
        int bad = parent < p.num_parents ? 0 : CARAT_DEV_BAD_CACHE_ID;
        int ctx = 0, last = 0, rows = 0, from = -1;
        const int fresh = p.new_pages[job];
        if (!bad) {
            ctx = p.context_lengths[parent];
            if (ctx < 0 || ctx > (long long)p.max_pages * p.page_rows) bad = CARAT_DEV_BAD_CONTEXT;
        }
        if (!bad) {
            last = ctx / p.page_rows;
            rows = ctx - last * p.page_rows;
            if (last < p.max_pages) from = p.page_table[(long long)parent * p.max_pages + last];
            if (fresh >= p.num_pages || (fresh >= 0 && rows > 0 && !page_ok(p, from)))
                bad = CARAT_DEV_BAD_CACHE_ID;
        }
        if (bad) {
            if (blockIdx.x == 0 && threadIdx.x == 0) set_status(p.dev_status, bad);
            continue;
        }
        if ((int)blockIdx.x <= 2 * p.pieces) {
            if (fresh >= 0) copy_piece(p, from, fresh, rows);
            continue;
        }
        const int32_t *line = p.page_table + (long long)parent * p.max_pages;
        int32_t *child = p.child_table + (long long)job * p.max_pages;
        for (int i = threadIdx.x; i < last; i += kCopyThreads) child[i] = line[i];
        if (threadIdx.x == 0) {
            if (last < p.max_pages) child[last] = fresh >= 0 ? fresh : from;
            if (p.child_lengths) p.child_lengths[job] = ctx;
        }
    }
}

// Whole pages, and in CTAs behind the copies' (blockIdx.x > 2 * pieces) the table: each
// entry that names a moved page is replaced, a thread an entry.  Copies and table do not
// depend on one another.
__global__ void __launch_bounds__(kCopyThreads) pages_move_kernel(const PagesParams p) {
    wait_for_prior_launch();
    let_next_launch_start();
    const int maps = (int)gridDim.x - (2 * p.pieces + 1);
    if ((int)blockIdx.x <= 2 * p.pieces) {
        for (int job = blockIdx.y; job < p.count; job += gridDim.y) {
            const int src = p.src[job], dst = p.dst[job];
            if (src < 0) continue;
            if (!page_ok(p, src) || !page_ok(p, dst)) {
                if (blockIdx.x == 0 && threadIdx.x == 0)
                    set_status(p.dev_status, CARAT_DEV_BAD_CACHE_ID);
                continue;
            }
            copy_piece(p, src, dst, p.page_rows);
        }
        return;
    }
    __shared__ int s_src[kMapSources];
    const long long mine = (blockIdx.x - (2 * p.pieces + 1)) + (long long)maps * blockIdx.y;
    const long long stride = (long long)maps * gridDim.y;
    for (long long base = mine * kCopyThreads; base < p.table_entries;
         base += stride * kCopyThreads) {
        const long long at = base + threadIdx.x;
        const int held = at < p.table_entries ? p.table[at] : -1;
        int found = -1;
        for (int first = 0; first < p.count; first += kMapSources) {
            const int n = min(kMapSources, p.count - first);
            __syncthreads();
            for (int i = threadIdx.x; i < n; i += kCopyThreads) s_src[i] = p.src[first + i];
            __syncthreads();
            for (int i = 0; i < n; ++i)
                if (s_src[i] == held) found = first + i;
        }
        if (held >= 0 && found >= 0 && page_ok(p, held)) {
            const int dst = p.dst[found];
            if (page_ok(p, dst)) p.table[at] = dst;
        }
    }
}

dim3 jobs_grid(int wide, int count) { return dim3(wide, count < 65535 ? count : 65535); }

}  // namespace

static PagesParams with_pieces(PagesParams p) {
    p.pieces = (int)((p.page_rows * p.row_bytes + kPieceBytes - 1) / kPieceBytes);
    return p;
}

cudaError_t launch_pages_copy(const PagesParams &call, cudaStream_t stream) {
    const PagesParams p = with_pieces(call);
    return launch_dependent(pages_copy_kernel, jobs_grid(2 * p.pieces + 1, p.count),
                            dim3(kCopyThreads), 0, stream, p);
}

cudaError_t launch_paged_fork(const PagesParams &call, cudaStream_t stream) {
    const PagesParams p = with_pieces(call);
    return launch_dependent(paged_fork_kernel, jobs_grid(2 * p.pieces + 2, p.count),
                            dim3(kCopyThreads), 0, stream, p);
}

cudaError_t launch_pages_move(const PagesParams &call, cudaStream_t stream) {
    const PagesParams p = with_pieces(call);
    const dim3 copies = jobs_grid(2 * p.pieces + 1, p.count);
    const long long blocks = (p.table_entries + kCopyThreads - 1) / kCopyThreads;
    const long long most = (blocks + copies.y - 1) / copies.y;
    return launch_dependent(pages_move_kernel,
                            dim3(copies.x + (int)(most < 1024 ? most : 1024), copies.y),
                            dim3(kCopyThreads), 0, stream, p);
}

}  // namespace carat
