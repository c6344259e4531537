// pool.cu -- host-side allocator of a shared HBM pool of KV pages.
//
// "Improving Decode Throughput on Intel Gaudi 3", "Our approach": the ring
// buffers of sliding-window layers are allocated in the same HBM that backs
// the global-attention KV pages, one shared pool, so that short requests can
// take more ring space and long requests more pages.  This allocator hands
// out page ids of one pool: a ring is an aligned run of `pages_per_ring`
// pages (its ring id is the first page / pages_per_ring, which is how the
// ring kernels address it), a global page is any single page.  Single pages
// are taken first from blocks that pages already broke up, then from the
// highest free block, so whole aligned blocks stay available for rings.
// A single page may have several owners (requests that share a beginning): it
// is free when as many have given it back.  Blocks that single pages broke up
// can be emptied again by moving their pages into free places elsewhere.
// Host code only; the device memory itself belongs to the caller.
#include <algorithm>
#include <cstdint>
#include <mutex>
#include <new>
#include <vector>

#include "carat_internal.cuh"

struct carat_pool {
    int num_pages = 0;
    int pages_per_ring = 0;
    int num_blocks = 0;
    std::vector<uint8_t> page_state;   // 0 free, 1 single page, 2 part of a ring
    std::vector<int> page_owners;      // owners of a single page
    std::vector<int> block_free;       // free pages per block
    std::vector<uint8_t> block_ring;   // block holds a ring
    int used_pages = 0;
    int used_rings = 0;
    std::mutex mutex;
};

namespace {

// Blocks: [b * ppr, (b + 1) * ppr) for b < num_blocks; pages past the last
// whole block can only be single pages.
int block_of(const carat_pool *p, int page) {
    const int b = page / p->pages_per_ring;
    return b < p->num_blocks ? b : -1;
}

}  // namespace

extern "C" {

carat_pool *carat_pool_create(int num_pages, int pages_per_ring) {
    if (num_pages < 1 || pages_per_ring < 1) return nullptr;
    carat_pool *p = new (std::nothrow) carat_pool;
    if (!p) return nullptr;
    p->num_pages = num_pages;
    p->pages_per_ring = pages_per_ring;
    p->num_blocks = num_pages / pages_per_ring;
    try {
        p->page_state.assign((size_t)num_pages, 0);
        p->page_owners.assign((size_t)num_pages, 0);
        p->block_free.assign((size_t)p->num_blocks, pages_per_ring);
        p->block_ring.assign((size_t)p->num_blocks, 0);
    } catch (...) {   // out of memory
        delete p;
        return nullptr;
    }
    return p;
}

void carat_pool_destroy(carat_pool *p) { delete p; }

int carat_pool_alloc_ring(carat_pool *p) {
    if (!p) return -1;
    std::lock_guard<std::mutex> lock(p->mutex);
    // lowest whole free block (single pages are taken from the top)
    for (int b = 0; b < p->num_blocks; ++b) {
        if (p->block_free[b] == p->pages_per_ring) {
            for (int i = 0; i < p->pages_per_ring; ++i) p->page_state[(size_t)b * p->pages_per_ring + i] = 2;
            p->block_free[b] = 0;
            p->block_ring[b] = 1;
            ++p->used_rings;
            return b;
        }
    }
    return -1;
}

int carat_pool_free_ring(carat_pool *p, int ring_id) {
    if (!p) return -1;
    std::lock_guard<std::mutex> lock(p->mutex);
    if (ring_id < 0 || ring_id >= p->num_blocks || !p->block_ring[ring_id]) return -1;
    for (int i = 0; i < p->pages_per_ring; ++i) p->page_state[(size_t)ring_id * p->pages_per_ring + i] = 0;
    p->block_free[ring_id] = p->pages_per_ring;
    p->block_ring[ring_id] = 0;
    --p->used_rings;
    return 0;
}

int carat_pool_alloc_pages(carat_pool *p, int n, int32_t *out_pages) {
    if (!p || n < 0 || (n > 0 && !out_pages)) return -1;
    std::lock_guard<std::mutex> lock(p->mutex);
    // all or nothing: count what single pages may use
    long long avail = 0;
    for (int b = 0; b < p->num_blocks; ++b)
        if (!p->block_ring[b]) avail += p->block_free[b];
    for (int pg = p->num_blocks * p->pages_per_ring; pg < p->num_pages; ++pg)
        avail += p->page_state[pg] == 0;
    if (avail < n) return -1;
    int got = 0;
    auto take = [&](int pg) {
        p->page_state[pg] = 1;
        p->page_owners[pg] = 1;
        const int b = block_of(p, pg);
        if (b >= 0) --p->block_free[b];
        out_pages[got++] = pg;
    };
    // 1. pages past the last whole block, 2. blocks already broken up by
    // single pages, 3. whole free blocks from the top
    for (int pg = p->num_blocks * p->pages_per_ring; pg < p->num_pages && got < n; ++pg)
        if (p->page_state[pg] == 0) take(pg);
    for (int b = p->num_blocks - 1; b >= 0 && got < n; --b) {
        if (p->block_ring[b] || p->block_free[b] == 0 || p->block_free[b] == p->pages_per_ring)
            continue;
        for (int i = 0; i < p->pages_per_ring && got < n; ++i) {
            const int pg = b * p->pages_per_ring + i;
            if (p->page_state[pg] == 0) take(pg);
        }
    }
    for (int b = p->num_blocks - 1; b >= 0 && got < n; --b) {
        if (p->block_ring[b] || p->block_free[b] != p->pages_per_ring) continue;
        for (int i = 0; i < p->pages_per_ring && got < n; ++i) take(b * p->pages_per_ring + i);
    }
    p->used_pages += got;
    return got;
}

int carat_pool_free_pages(carat_pool *p, int n, const int32_t *pages) {
    if (!p || n < 0 || (n > 0 && !pages)) return -1;
    std::lock_guard<std::mutex> lock(p->mutex);
    // all or nothing: every entry must be an allocated single page, listed once
    for (int i = 0; i < n; ++i) {
        const int pg = pages[i];
        if (pg < 0 || pg >= p->num_pages || p->page_state[pg] != 1) {
            for (int x = 0; x < i; ++x) p->page_state[pages[x]] = 1;
            return -1;
        }
        p->page_state[pg] = 3;  // marked for release
    }
    for (int i = 0; i < n; ++i) {
        const int pg = pages[i];
        if (--p->page_owners[pg] > 0) {   // others still hold it
            p->page_state[pg] = 1;
            continue;
        }
        p->page_state[pg] = 0;
        const int b = block_of(p, pg);
        if (b >= 0) ++p->block_free[b];
        --p->used_pages;
    }
    return 0;
}

int carat_pool_share_pages(carat_pool *p, int n, const int32_t *pages) {
    if (!p || n < 0 || (n > 0 && !pages)) return -1;
    std::lock_guard<std::mutex> lock(p->mutex);
    for (int i = 0; i < n; ++i)
        if (pages[i] < 0 || pages[i] >= p->num_pages || p->page_state[pages[i]] != 1 ||
            p->page_owners[pages[i]] > 0x7fffffff - n)
            return -1;
    for (int i = 0; i < n; ++i) ++p->page_owners[pages[i]];
    return 0;
}

int carat_pool_plan_compaction(carat_pool *p, int max_moves, int32_t *out_src, int32_t *out_dst) {
    if (!p || max_moves < 0 || (max_moves > 0 && (!out_src || !out_dst))) return -1;
    std::lock_guard<std::mutex> lock(p->mutex);
    const int ppr = p->pages_per_ring;
    // blocks that hold single pages, the fullest first: a block is emptied from the back
    // of this list into the pages past the last block and into the blocks at its front
    std::vector<int> order;
    try {
        for (int b = 0; b < p->num_blocks; ++b)
            if (!p->block_ring[b] && p->block_free[b] < ppr) order.push_back(b);
    } catch (...) {
        return -1;
    }
    std::sort(order.begin(), order.end(), [&](int a, int b) {
        return p->block_free[a] != p->block_free[b] ? p->block_free[a] < p->block_free[b] : a > b;
    });
    long long room = 0;
    for (int pg = p->num_blocks * ppr; pg < p->num_pages; ++pg) room += p->page_state[pg] == 0;
    for (int b : order) room += p->block_free[b];
    int moves = 0, next = p->num_blocks * ppr;
    size_t into = 0;   // order[into]: the block being filled, once the tail is full
    int filled = -1;   // the last such block that a page was moved into
    auto free_place = [&](size_t last) -> int {
        for (; next < p->num_pages; ++next)
            if (p->page_state[next] == 0) return next;
        for (; into < last; ++into)
            for (int i = 0; i < ppr; ++i)
                if (p->page_state[order[into] * ppr + i] == 0) {
                    filled = (int)into;
                    return order[into] * ppr + i;
                }
        return -1;
    };
    for (size_t last = order.size(); last-- > 0;) {
        if ((int)last <= filled) break;   // it holds pages that were moved here
        const int b = order[last], used = ppr - p->block_free[b];
        room -= p->block_free[b];   // its own free places do not count
        if (room < used || moves + used > max_moves) break;
        for (int i = 0; i < ppr; ++i) {
            const int from = b * ppr + i;
            if (p->page_state[from] != 1) continue;
            const int to = free_place(last);
            if (to < 0) return moves;   // not reached: room was counted
            p->page_state[to] = 1;
            p->page_owners[to] = p->page_owners[from];
            p->page_state[from] = 0;
            p->page_owners[from] = 0;
            if (block_of(p, to) >= 0) --p->block_free[block_of(p, to)];
            ++p->block_free[b];
            out_src[moves] = from;
            out_dst[moves++] = to;
            --room;
        }
    }
    return moves;
}

int carat_pool_stats(carat_pool *p, int32_t *out4) {
    if (!p || !out4) return -1;
    std::lock_guard<std::mutex> lock(p->mutex);
    int whole = 0;
    for (int b = 0; b < p->num_blocks; ++b) whole += p->block_free[b] == p->pages_per_ring;
    out4[0] = p->num_pages - p->used_pages - p->used_rings * p->pages_per_ring;  // free pages
    out4[1] = whole;                                                             // whole free blocks
    out4[2] = p->used_rings;
    out4[3] = p->used_pages;
    return 0;
}

}  // extern "C"
