// paged_chunk.cu -- attention of a chunk of new tokens over bf16 pages.
//
// Query j of request b sits at position p = context_lengths[b] + j and sees key t when
//   t <= p  and  (window == 0  or  t > p - window  or  t < sinks);
//   out = sum_t softmax_t(scale q . k_t) v_t over the keys it sees.
//
// Rows.  The query heads that share a KV head and the chunk's tokens form rows r = j*g + h'
// (g = q_heads / kv_heads); a CTA holds the 128 / g tokens whose rows fill 128, a pair of
// CTAs (a cluster of two SMs) twice as many, and each key tile of 128 keys is loaded once
// for the pair, half by each:
//     S [256 rows x 128 keys] = Q . K_tile^T      A: own 128 rows, B: 64 keys a CTA
//     O [256 rows x 256 d]   += P . V_tile        A: own rows of P, B: 128 d a CTA
// tcgen05.mma cta_group::2, bf16 operands, fp32 accumulators.  Tensor memory of a CTA: O 256
// columns, two S tiles of 128; P (bf16) takes the place of the S tile it comes from and is
// read from there.  At head_dim 512 O of 128 rows would fill all 512 columns, so a pair
// takes one half of the value dimensions and the scores are computed for each half again
// (1.5 times the operations).
//
// What bounds it: the tensor pipe, where rows are many.  A pair reads K and V tiles at 32
// bytes a cycle and SM from L2, against 64 without pairs, which L2 could not give.  Measured:
// 8191 tokens of 16 heads over 8 of 256, 288 us, 1910 TFLOP/s (the library's product reaches
// 1917); over 2 of 512, 817 us, 1345 TFLOP/s of what is asked for and 2017 with the scores
// computed twice.  (A few replays; in a long stream of calls the power limit makes the latter
// 915 to 932, as the library's product falls to 1703.)  Under a window an item is short (9 tiles
// at a window of 1024) and its ends show: 8192 tokens 101 us, 1270 TFLOP/s.  There from the last
// product of an item to the first of the next 6000 to 7000 cycles pass, where a tile takes 2150:
// its output 2500 to 3700 (64 KB a CTA leave at about 32 bytes a cycle), the next scores' way to
// the softmax, 1500 for their weights.  Storing with the copy engine from shared memory, and
// finding the next item during the present one, changed that case and the others by 1% and cost
// short calls up to 7%; the output on warps of its own cost 18%.
//
// Softmax.  Two threads a row, 64 keys of a tile each in registers.  The running maximum is
// replaced only when a tile exceeds it by more than 8 (log2 units), so O is rarely read
// back and rescaled; P <= 2^8.  P is rounded to bf16 (the tensor core's operand, with V
// bf16; 2^-8 of each weight) and the rounded weights are summed, so numerator and
// denominator see the same ones.
//
// Keys.  An item (request, KV head, row tile, value half, split) walks the tiles that hold
// a key some row of the pair sees: those of the sinks, then from the first row's window to
// the last row's position.  A tile some row sees only in part is masked by position.  Its
// V rows could carry what no row may see into O through 0 x infinity: two warps look
// through such a tile's V for values that are not finite and zero those rows, and
// rows behind the last key, before the product; a row that sees such a key is written as
// NaN.
//
// Few items: their key tiles are split over CTA pairs, each piece leaves (max, sum,
// unnormalised O) and a second launch merges them.  How long a piece is goes by the
// lengths on the device: the pieces are alike and their number fits the pairs, whether one
// long request is among short ones or not.
//
// Schedule.  The grid has a CTA pair for every item, up to a few times the pairs that fit;
// a pair that has finished takes over the work of one that has not been launched (cluster
// launch control), so the items, of very different lengths under masks, windows and counts,
// go to whoever is free.  The producer asks, finds the item and hands it to the other roles
// through a ring of four.  The next item's keys and queries are loaded and its first scores
// computed while the last one's output leaves.  Code that runs once an item is kept short
// (rolled loops, one copy): it comes from a cold instruction cache, and an unrolled output
// of the same work took 5000 cycles.
//
// Warp roles (384 threads): warp 0 TMA producer (each CTA its own halves, counted on the
// leader's barriers), warp 1 of the leader issues the products, warps 2-3 look through V,
// warps 4-11 softmax, rescale and output (one thread a row took 1.9 us a tile at head_dim
// 256, nearly twice the products' time).  Every wait is bounded: on a timeout
// CARAT_DEV_TIMEOUT is set and the CTA stops, waits for its own copies and products, and
// returns.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <cmath>

#include <cuda_bf16.h>

#include "carat_internal.cuh"
#include "tc_common.cuh"
#include "tma_host.h"

namespace carat {
namespace {

constexpr int kKeys = 128;              // keys of a tile
constexpr int kRows = 128;              // rows of a CTA
constexpr int kDV = 256;                // value dimensions of an item
constexpr int kStage = 32768;           // K: 64 keys x 256 d, or V: 128 keys x 128 d
constexpr int kThreads = 384, kSoftmax = 256;
constexpr int kJobs = 4;                // items handed to the other roles
constexpr int kPieceCost = 3;           // of a piece besides its key tiles, in key tiles
constexpr int kMergeCost = 4;           // of the merge of what was split, in key tiles
constexpr int kUnits = 8;               // CTA pairs of the grid, times the pairs that fit
constexpr int kMasked = 8;              // masked tiles of an item: 3 + 3 + 1 at most
constexpr int kRecords = 5;             // items whose masked tiles' V is on record
constexpr uint32_t kInTurn = 3;         // masked tiles whose V is on its way
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kSlack = 8.0f;          // log2 units
// Maxima from which on a score is rounded before the maximum is taken from it.  Below, the
// two are one fused operation whose exact product differs from the rounded maximum by half a
// unit of its last place, the same for the whole row: a factor of 2^(1/2) at most, which numerator
// and denominator share.  From 2^31 on it would leave the range of a float.
constexpr float kRounded = 16777216.f;  // 2^24

template <int D>
struct Lay {
    static constexpr int KST = D / 256;                 // stages of a K tile
    // Stage ring; five stages at head_dim 256 were no faster (323 us against 290, 8191 tokens).
    static constexpr int NS = D == 256 ? 4 : 3;
    static constexpr int kSlab = kRows * 128;           // 64 d of Q
    static_assert(NS <= 4, "the records of masked tiles and their barriers count on it");
    static constexpr int kOffQ = NS * kStage;
    static constexpr int kOffOut = D == 512 ? kOffQ : kOffQ + D / 64 * kSlab;
    // The output's way out: 32 rows of 128 bytes a softmax warp.  At head_dim 512 the place
    // is the queries', and the next item's queries are loaded behind it.
    static constexpr bool kOutInQ = D == 512;
    static constexpr int kOffMisc = kOffQ + D / 64 * kSlab + (kOutInQ ? 0 : 8 * 4096);
    static constexpr int kMisc = 2560;
    static constexpr int kAlloc = kOffMisc + kMisc;
    static_assert(kAlloc <= 232448, "more dynamic shared memory than one CTA may use");
};

struct Request {
    long long ctx;
    int n;
};

__device__ __forceinline__ Request load_request(const PagedChunkParams &p, int b) {
    return {p.context_lengths[b], p.new_counts ? p.new_counts[b] : p.k};
}

__device__ __forceinline__ bool request_ok(const PagedChunkParams &p, const Request &r) {
    return r.ctx >= 0 && r.n >= 0 && r.n <= p.k && r.ctx + r.n <= p.capacity;
}

struct Plan {
    int tokens;      // of a CTA
    int halves;      // value halves
    int splits;      // most pieces of an item
    int by_length;   // how many goes by the requests' lengths (else all have `splits`)
    int units;       // CTA pairs of the grid: pair u has the items u, u + units, ...
    float2 *part_ml; // [B k Hq][splits]
    float *part_o;   // [B k Hq][splits][D]
    int *pieces;     // [B] pieces of a request's items
};

// Key tiles of the rows at positions [lo, hi]: the sinks', then the window's.  Positions
// are below 2^31 (a request's capacity).
struct Keys {
    int lo, hi;
    int first;              // the window's first tile
    int sink_tiles, count;

    Keys() = default;
    __device__ __forceinline__ Keys(const PagedChunkParams &p, int lo_, int hi_)
        : lo(lo_), hi(hi_) {
        first = p.window > 0 && lo - p.window + 1 > 0 ? (lo - p.window + 1) / kKeys : 0;
        sink_tiles = p.window > 0 && p.sinks > 0 ? min((p.sinks - 1) / kKeys + 1, first) : 0;
        count = sink_tiles + hi / kKeys - first + 1;
    }
    __device__ __forceinline__ int base(int x) const {
        return (x < sink_tiles ? x : first + x - sink_tiles) * kKeys;
    }
    // whether some row sees some key of the tile at t0 and not another
    __device__ __forceinline__ bool masked(const PagedChunkParams &p, int t0) const {
        if (t0 + (kKeys - 1) > lo) return true;
        return p.window > 0 && t0 <= hi - p.window && t0 + (kKeys - 1) >= p.sinks;
    }
};

// Pieces of `count` tiles: split s takes [count s / splits, count (s + 1) / splits).
// (Fewer than 2^24 tiles, fewer splits than SMs: the product fits 32 bits.)
__device__ __forceinline__ int split_at(int count, int s, int splits) {
    return splits == 1 ? count * s : (int)((uint32_t)count * (uint32_t)s / (uint32_t)splits);
}

// One pair's share of a request's chunk for one KV head.
struct Item {
    int b, c, vh, split, splits;
    int j0, n, ctx;        // the pair's first token; the request's tokens, and before them
};

// Row tiles of a request, and key tiles of the last (the longest).
struct Load {
    int rows, keys;
};
__device__ __forceinline__ Load load_of(const PagedChunkParams &p, const Plan &plan,
                                        const Request &rq) {
    if (!request_ok(p, rq) || rq.n == 0) return {0, 0};
    const int span = 2 * plan.tokens, rows = (rq.n + span - 1) / span;
    return {rows, Keys(p, (int)rq.ctx + (rows - 1) * span, (int)rq.ctx + rq.n - 1).count};
}

// Pieces of an item that has this many key tiles.
__device__ __forceinline__ int pieces_of(const Plan &plan, int keys, int length) {
    return min(plan.splits, max(1, (keys + length - 1) / length));
}

// Key tiles of a piece where requests differ, by a whole warp: of 32 lengths between a
// quarter of and nearly four times a pair's share of all tiles, the one whose rounds of pieces
// take the least, a piece costing its tiles and kPieceCost for its start and its output, and
// the merge kMergeCost.  Requests of which none is longer than a pair's share by more than
// those costs are left whole without a search.
__device__ __noinline__ int piece_length(const PagedChunkParams &p, const Plan &plan, int lane) {
    const int per_tile = p.kv_heads * plan.halves;
    float total = 0.f;
    int most = 0;
    Load held{};
    for (int base = 0; base < p.batch; base += 32) {
        held = {0, 0};
        if (base + lane < p.batch) held = load_of(p, plan, load_request(p, base + lane));
        total += (float)held.rows * held.keys;
        most = max(most, held.keys);
    }
    most = __reduce_max_sync(kFull, most);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
    const float share = total * per_tile / plan.units;
    if (most <= share + (kPieceCost + kMergeCost)) return max(most, 1);
    const int length = max(1, (int)(fast_exp2((lane - 16) * 0.125f) * share + 0.5f));
    int count = 0, whole = 0, longest = 0;
    for (int base = 0; base < p.batch; base += 32) {
        if (p.batch > 32) {
            held = {0, 0};
            if (base + lane < p.batch) held = load_of(p, plan, load_request(p, base + lane));
        }
        for (int i = 0; i < min(32, p.batch - base); ++i) {
            const int rows = __shfl_sync(kFull, held.rows, i);
            const int keys = __shfl_sync(kFull, held.keys, i);
            if (rows == 0) continue;
            const int n = pieces_of(plan, keys, length);
            count += rows * n;
            whole += rows;
            longest = max(longest, (keys + n - 1) / n);
        }
    }
    const float cost = (float)((count * per_tile + plan.units - 1) / plan.units) *
                           (longest + kPieceCost) +
                       (count > whole ? kMergeCost : 0);
    float best = cost;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = fminf(best, __shfl_xor_sync(kFull, best, o));
    return __shfl_sync(kFull, length, __ffs(__ballot_sync(kFull, cost == best)) - 1);
}

// The items in order, request after request, found by a whole warp.  Requests are looked at
// 32 at a time, one a lane.
struct Items {
    int length = 0;        // key tiles of a piece (items are split)
    int base = -32;        // first request held
    int upto = 0;          // items of the held requests up to this lane's, and before
    int before = 0;        // items before the held requests
    int n = 0, tiles = 0, ctx = 0, splits = 1;   // this lane's request

    // Item number id, or false: there are fewer.
    __device__ __forceinline__ bool find(const PagedChunkParams &p, const Plan &plan, int lane,
                                         int id, Item &it) {
        const int per_split = p.kv_heads * plan.halves;
        if (plan.by_length && length == 0) {
            // Requests alike: as many pieces as pairs, in one round.  (The search takes about
            // 3 us.)
            Load held{};
            if (lane < p.batch) held = load_of(p, plan, load_request(p, lane));
            const int keys = __reduce_max_sync(kFull, held.keys);
            const int rows = __reduce_add_sync(kFull, held.rows);
            if (p.batch <= 32 && __all_sync(kFull, held.rows == 0 || held.keys == keys)) {
                const int pieces = min(plan.splits, max(1, plan.units / max(1, rows * per_split)));
                length = max(1, (keys + pieces - 1) / pieces);
            } else {
                length = piece_length(p, plan, lane);
            }
        }
        if (id < before) {
            base = -32;
            before = 0;
        }
        while (true) {
            const unsigned hit = __ballot_sync(kFull, base >= 0 && id < upto);
            if (hit) {
                const int src = __ffs(hit) - 1;
                const int t_src = __shfl_sync(kFull, tiles, src);
                it.splits = __shfl_sync(kFull, splits, src);
                const int per_tile = per_split * it.splits;
                int rest = id - (__shfl_sync(kFull, upto, src) - t_src * per_tile);
                it.b = base + src;
                it.n = __shfl_sync(kFull, n, src);
                it.ctx = __shfl_sync(kFull, ctx, src);
                const int tile = t_src - 1 - rest / per_tile;   // the longest first
                rest %= per_tile;
                it.split = rest % it.splits;
                rest /= it.splits;
                it.vh = rest % plan.halves;
                it.c = rest / plan.halves;
                it.j0 = tile * 2 * plan.tokens;
                return true;
            }
            if (base + 32 >= p.batch) return false;
            if (base >= 0) before = __shfl_sync(kFull, upto, 31);
            base += 32;
            tiles = 0;
            splits = 1;
            if (base + lane < p.batch) {
                const Request rq = load_request(p, base + lane);
                ctx = (int)rq.ctx;
                n = rq.n;
                const Load load = load_of(p, plan, rq);
                tiles = load.rows;
                splits = plan.by_length ? pieces_of(plan, load.keys, length) : plan.splits;
            }
            upto = tiles * per_split * splits;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, upto, o);
                if (lane >= o) upto += y;
            }
            upto += before;
        }
    }
};

// One item's split: its tiles in the order they are taken, from the first that every row
// sees whole, so that no row's first maximum is that of a few keys (the maxima then rise
// past the slack tile after tile, 1200 to 1700 cycles each time), round to those before it.
// n = 0: no item left, and it.b says whether this pair writes the rejected requests.
struct Job {
    Item it;
    Keys keys;
    int x0, n, turn;

    __device__ __forceinline__ int base(int x) const {
        const int y = x + turn;
        return keys.base(x0 + (y >= n ? y - n : y));
    }
};

__device__ __forceinline__ Job job_of(const PagedChunkParams &p, const Plan &plan, const Item &it) {
    Job j;
    j.it = it;
    j.keys = Keys(p, it.ctx + it.j0, it.ctx + min(it.j0 + 2 * plan.tokens, it.n) - 1);
    j.x0 = split_at(j.keys.count, it.split, it.splits);
    j.n = split_at(j.keys.count, it.split + 1, it.splits) - j.x0;
    j.turn = 0;
    while (j.turn < j.n && j.keys.masked(p, j.keys.base(j.x0 + j.turn))) ++j.turn;
    if (j.turn >= j.n) j.turn = 0;
    return j;
}

template <int NS>
struct Shared {
    uint64_t full[NS];      // leader: a stage's bytes of both CTAs have landed
    uint64_t empty[NS];     // both: the products that read the stage are done
    uint64_t q_full;        // leader
    uint64_t q_empty;       // both: an item's last scores are computed (and its output has left)
    uint64_t s_full[2];     // both: a tile's scores are in tensor memory
    uint64_t p_full[2];     // leader: its weights are
    uint64_t pv_done[2];    // both: a tile's value product is done (tiles in turn)
    // Masked tiles in turn.  The third next one's V is loaded four loads later or more, when
    // this one's product is done; the second next one's can be three later (an item's last
    // two V's follow one another, an item of one tile has one K before its V).
    uint64_t v_ready[kInTurn];   // each CTA's own: its half of the tile's V has landed
    uint64_t v_clean[kInTurn];   // leader: both halves are looked through
    uint64_t drain;
    uint64_t job_full[kJobs], job_empty[kJobs];   // each CTA's own
    uint64_t answered[kJobs];                     // each CTA's own
    uint64_t answer_read[kJobs];                  // leader: the other CTA has read its answer
    alignas(16) uint4 answer[kJobs];              // which cluster's work is taken over
    uint32_t tmem;
    int abort_flag;
    Job job[kJobs];
    // Keys of masked tiles with values that are not finite, of kRecords items with such tiles
    // in turn.  V of a tile lands when the products have used what its stage held, at most
    // four loads before it, and a tile is two loads or more.  So while a CTA's warps have not
    // said that the first such tile of item M (of these) is looked through, the other's are
    // at item M + 1 at most; and the softmax warps are past item M - 3, as the products are
    // past all of M - 2.  At that tile the record of M + 2, which was that of M - 3, is cleared.
    uint32_t poison[kRecords];
    uint32_t bad[kRecords][kMasked][4];
    // A row's two threads tell each other.  They change places every time: each writes over
    // what the other told last, which it alone has read.
    float row[2][kRows];
};

// Bounded wait; false on a timeout or when another role of this CTA gave up.  kCluster:
// what threads of the other CTA wrote before they released the barrier is seen.
template <bool kCluster>
__device__ __forceinline__ bool passed(uint64_t *bar, uint32_t parity) {
    return kCluster ? tc::mbar_try_wait_cluster(bar, parity) : tc::mbar_try_wait(bar, parity);
}

template <bool kCluster>
__device__ __noinline__ bool wait_on(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                     int *dev_status) {
    const uint64_t t0 = tc::globaltimer_ns();
    for (uint32_t round = 1;; ++round) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (passed<kCluster>(bar, parity)) return true;
        if (*abort_flag) return false;
        if (tc::wait_expired(t0, round, 2000000000ull)) {
            *abort_flag = 1;
            set_status(dev_status, CARAT_DEV_TIMEOUT);
            return false;
        }
    }
}

// A whole warp goes on or stops as one.
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity,
                                          volatile int *abort_flag, int *dev_status) {
    const bool ok =
        passed<kCluster>(bar, parity) || wait_on<kCluster>(bar, parity, abort_flag, dev_status);
    return __all_sync(kFull, ok) != 0;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Bits [0, n) of 64, any n.
__device__ __forceinline__ uint64_t low_bits(int n) {
    return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1ull;
}

// The two warps that share 32 rows meet; whether one of them has to stop, so that both do.
__device__ __forceinline__ bool rows_barrier(int quad, bool stop) {
    uint32_t out;
    asm volatile(
        "{\n\t.reg .pred pin, pout;\n\t"
        "setp.ne.u32 pin, %1, 0;\n\t"
        "bar.red.or.pred pout, %2, 64, pin;\n\t"
        "selp.u32 %0, 1, 0, pout;\n\t}"
        : "=r"(out)
        : "r"((uint32_t)stop), "r"(1 + quad)
        : "memory");
    return out != 0;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    paged_chunk_kernel(const __grid_constant__ PagedChunkParams p, const Plan plan,
                       const __grid_constant__ CUtensorMap map_q,
                       const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v) {
    using L = Lay<D>;
    constexpr int NS = L::NS, KST = L::KST;
    extern __shared__ __align__(1024) uint8_t smem[];
    auto *sh = reinterpret_cast<Shared<NS> *>(smem + L::kOffMisc);
    static_assert(sizeof(Shared<NS>) <= L::kMisc, "misc area");
    uint8_t *s_q = smem + L::kOffQ;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = (int)tc::cluster_ctarank(), pair = blockIdx.x / 2;

    if (threadIdx.x == 96) {
        tc::tma_prefetch_map(&map_q);
        tc::tma_prefetch_map(&map_k);
        tc::tma_prefetch_map(&map_v);
        for (int i = 0; i < NS; ++i) {
            tc::mbar_init(&sh->full[i], 1);
            tc::mbar_init(&sh->empty[i], 1);
        }
        tc::mbar_init(&sh->q_full, 1);
        tc::mbar_init(&sh->q_empty, L::kOutInQ ? 9 : 1);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sh->s_full[i], 1);
            tc::mbar_init(&sh->p_full[i], 16);
            tc::mbar_init(&sh->pv_done[i], 1);
        }
        for (int i = 0; i < kInTurn; ++i) {
            tc::mbar_init(&sh->v_ready[i], 1);
            tc::mbar_init(&sh->v_clean[i], 4);
        }
        for (int i = 0; i < kRecords; ++i) sh->poison[i] = 0;
        tc::mbar_init(&sh->drain, 1);
        for (int i = 0; i < kJobs; ++i) {
            tc::mbar_init(&sh->job_full[i], 1);
            tc::mbar_init(&sh->answered[i], 1);
            tc::mbar_init(&sh->answer_read[i], 1);
            tc::mbar_init(&sh->job_empty[i], rank == 0 ? 11 : 10);
        }
        tc::fence_mbar_init();
        sh->abort_flag = 0;
    }
    if (threadIdx.x < kRecords * kMasked * 4) (&sh->bad[0][0][0])[threadIdx.x] = 0;
    if (warp == 1) {
        tc::tmem_alloc_pair(&sh->tmem, 512);
        tc::tmem_relinquish_pair();
    }
    wait_for_prior_launch();
    let_next_launch_start();
    // The first item is looked up while the barriers and tensor memory are made ready.
    Items list;
    Item it{};
    bool found = false;
    if (warp == 0) found = list.find(p, plan, lane, pair, it);
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_arrive();
    tc::cluster_wait();
    tc::tc_fence_after();
    const uint32_t tmem = sh->tmem;
    const uint32_t t_o = tmem, t_s = tmem + kDV;
    volatile int *abort_flag = &sh->abort_flag;
    // Every role but the producer: the next item, or false (none left, or a wait ran out).
    uint32_t taken = 0;
    auto take = [&](bool &alive) -> const Job * {
        const int slot = taken % kJobs;
        alive = alive &&
                warp_wait(&sh->job_full[slot], (taken / kJobs) & 1, abort_flag, p.dev_status);
        ++taken;
        return alive && sh->job[slot].n > 0 ? &sh->job[slot] : nullptr;
    };
    auto give_back = [&]() {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh->job_empty[(taken - 1) % kJobs]);
    };

    if (warp == 0) {
        // ---------------------------------------------------------------- producer
        uint32_t cnt = 0, items = 0, masked_v = 0;   // stages, items, V of masked tiles
        bool alive = true;
        const uint32_t q_bytes = plan.tokens * p.group * 128;
        uint32_t published = 0, asked = 0;
        // Both CTAs' producers get the same answers, the leader asks.  An answer's place is
        // used again after kJobs more, once the other CTA has read it there: work taken over
        // that turns out to be none (a padded batch) goes through no other ring, and the
        // other CTA may still wait for its queries' place.
        int unit = pair, id = pair;
        bool pending = false, rejects = pair == 0;
        auto ask = [&]() {
            const int slot = asked % kJobs;
            if (rank == 0 && asked >= kJobs)
                alive = warp_wait<true>(&sh->answer_read[slot], ((asked / kJobs) & 1) ^ 1,
                                        abort_flag, p.dev_status);
            if (!alive) return;
            if (lane == 0) {
                tc::fence_proxy_async_smem();
                tc::mbar_arrive_expect_tx(&sh->answered[slot], 16);
                if (rank == 0) tc::ask_for_cluster(&sh->answer[slot], &sh->answered[slot]);
            }
            __syncwarp();
            pending = true;
        };
        for (bool first = true; alive; first = false) {
            Job tiles{};
            if (unit >= 0) {
                if (!first) found = list.find(p, plan, lane, id, it);
                if (!found) {
                    // this pair's work is done: another's
                    const int slot = asked % kJobs;
                    if (!pending) ask();
                    alive = alive && warp_wait(&sh->answered[slot], (asked / kJobs) & 1, abort_flag,
                                               p.dev_status);
                    if (!alive) break;
                    const int taken_over = tc::cluster_taken(&sh->answer[slot]);
                    __syncwarp();
                    if (rank == 1 && lane == 0) {
                        tc::fence_proxy_async_smem();
                        tc::mbar_arrive_cluster(tc::map_to_rank(&sh->answer_read[slot], 0));
                    }
                    ++asked;
                    pending = false;
                    unit = id = taken_over < 0 ? -1 : taken_over / 2;
                    rejects |= unit == 0;
                    continue;
                }
                id += plan.units;
                // for the merge (a request's last rows have a tile in every piece)
                if (plan.splits > 1 && it.split == 0 && lane == 0) plan.pieces[it.b] = it.splits;
                tiles = job_of(p, plan, it);
                if (tiles.n == 0) continue;
            }
            const int slot = published % kJobs;
            if (published >= kJobs)
                alive = warp_wait(&sh->job_empty[slot], ((published / kJobs) & 1) ^ 1, abort_flag,
                                  p.dev_status);
            if (!alive) break;
            if (unit < 0) tiles.it.b = rejects;
            if (lane == 0) {
                sh->job[slot] = tiles;
                tc::mbar_arrive(&sh->job_full[slot]);
            }
            ++published;
            if (unit < 0) break;
            const int n = tiles.n;
            int row_held = 0;   // lane l: pool row of the item's tile 32 * (x / 32) + l
            auto fetch = [&](int x) {
                if (x + lane < n) {
                    const int t = tiles.base(x + lane), at = t / p.page_rows;
                    const int page = p.page_table[(size_t)it.b * p.max_pages + at];
                    if (page < 0 || page >= p.num_pages) {
                        set_status(p.dev_status, CARAT_DEV_BAD_CACHE_ID);
                        row_held = -1;
                    } else {
                        row_held = page * p.page_rows + (t - at * p.page_rows);
                    }
                }
            };
            auto load = [&](bool is_v, int row, int part, bool masked) {
                const int s = cnt % NS;
                if (cnt >= NS && alive)
                    alive = warp_wait(&sh->empty[s], ((cnt / NS) & 1) ^ 1, abort_flag, p.dev_status);
                if (!alive) return;
                if (lane == 0) {
                    // V of a masked tile is counted by each CTA for itself, so that it is looked
                    // through as soon as it is there (the products wait for that, not for the
                    // bytes): waiting for the products' warp to come to it cost 1700 cycles.
                    uint64_t *own = &sh->v_ready[masked_v % kInTurn];
                    if (masked) {
                        tc::mbar_arrive_expect_tx(own, kStage);
                        if (rank == 0) tc::mbar_arrive(&sh->full[s]);
                    } else if (rank == 0) {
                        tc::mbar_arrive_expect_tx(&sh->full[s], 2 * kStage);
                    }
                    const uint32_t bar = masked ? tc::map_to_rank(own, rank)
                                                : tc::map_to_rank(&sh->full[s], 0);
                    // a page outside the pool: rows behind the tensor's end read as zeros
                    const int at =
                        row < 0 ? p.num_pages * p.page_rows : row + (is_v ? 0 : rank * 64);
                    if (is_v)
                        tc::tma_load_4d_pair(smem + s * kStage, &map_v, 0, at, it.vh * 4 + rank * 2,
                                             it.c, bar);
                    else
                        tc::tma_load_4d_pair(smem + s * kStage, &map_k, 0, at, part * 4, it.c, bar);
                }
                ++cnt;
                masked_v += masked;
            };
            int prev = 0;
            for (int x = 0; x <= n && alive; ++x) {
                int row = 0;
                if (x < n) {
                    if ((x & 31) == 0) fetch(x);
                    row = __shfl_sync(kFull, row_held, x & 31);
                    for (int k = 0; k < KST; ++k) load(false, row, k, false);
                }
                if (x == 0 && alive) {
                    // the queries' place is free when the last item's last scores are computed
                    if (items > 0)
                        alive = warp_wait(&sh->q_empty, (items - 1) & 1, abort_flag, p.dev_status);
                    if (alive && lane == 0) {
                        if (rank == 0) tc::mbar_arrive_expect_tx(&sh->q_full, 2 * (D / 64) * q_bytes);
                        const uint32_t bar = tc::map_to_rank(&sh->q_full, 0);
                        for (int i = 0; i < D / 64; ++i)
                            tc::tma_load_4d_pair(s_q + i * L::kSlab, &map_q, i * 64, it.c * p.group,
                                                 it.j0 + rank * plan.tokens, it.b, bar);
                    }
                    if (alive) ++items;
                }
                if (x > 0) load(true, prev, 0, tiles.keys.masked(p, tiles.base(x - 1)));
                prev = row;
                if (x == 0 && !pending && alive) ask();   // for the work after this
            }
        }
        // An answer that is still on its way lands before anyone leaves, and what both CTAs'
        // copies still carry.
        if (!alive && pending) tc::mbar_wait(&sh->answered[asked % kJobs], (asked / kJobs) & 1);
        for (uint32_t i = masked_v > kInTurn ? masked_v - kInTurn : 0; !alive && i < masked_v; ++i)
            tc::mbar_wait(&sh->v_ready[i % kInTurn], (i / kInTurn) & 1);
        if (!alive && rank == 0) {
            if (items > 0) tc::mbar_wait(&sh->q_full, (items - 1) & 1);
            for (uint32_t i = cnt > NS ? cnt - NS : 0; i < cnt; ++i)
                tc::mbar_wait(&sh->full[i % NS], (i / NS) & 1);
        }
    } else if (warp == 1 && rank == 0) {
        // ---------------------------------------------------------------- products
        const uint32_t id_qk = tc::idesc_bf16_f32(256, kKeys, false, false) |
                               (p.scale_log2 < 0.f ? 1u << 13 : 0u);   // negates A
        constexpr uint32_t id_pv = tc::idesc_bf16_f32(256, kDV, false, true);
        const uint32_t q_addr = tc::smem_u32(s_q), st_addr = tc::smem_u32(smem);
        uint32_t cnt = 0, items = 0, g = 0, vcnt = 0;   // stages, items, tiles, masked tiles
        bool alive = true;
        const uint64_t q_desc = tc::sdesc_sw128(q_addr, 16, 1024);
        const uint64_t k_desc = tc::sdesc_sw128(st_addr, 16, 1024);
        const uint64_t v_desc = tc::sdesc_sw128(st_addr, 16384, 1024);
        while (const Job *job = take(alive)) {
            const Job tiles = *job;
            give_back();
            const int n = tiles.n;
            alive = warp_wait(&sh->q_full, items & 1, abort_flag, p.dev_status);
            ++items;
            for (int x = 0; x <= n && alive; ++x) {
                if (x < n) {
                    const uint32_t buf = (g + x) & 1;
                    for (int k = 0; k < KST; ++k, ++cnt) {
                        const int s = cnt % NS;
                        alive = warp_wait(&sh->full[s], (cnt / NS) & 1, abort_flag, p.dev_status);
                        if (!alive) break;
                        tc::tc_fence_after();
                        // Unrolled: four at a time cost 8% of the whole call.  (Addresses in
                        // descriptors count 16 bytes.)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            tc::mma_bf16_ss_pair(
                                t_s + buf * kKeys,
                                q_desc + ((k * 4 + i / 4) * (L::kSlab / 16) + (i & 3) * 2),
                                k_desc + (s * (kStage / 16) + i / 4 * 512 + (i & 3) * 2), id_qk,
                                k > 0 || i > 0);
                        tc::mma_commit_pair(&sh->empty[s]);
                    }
                    if (!alive) break;
                    tc::mma_commit_pair(&sh->s_full[buf]);
                    if (x == n - 1) tc::mma_commit_pair(&sh->q_empty);
                }
                if (x == 0) continue;
                const int y = x - 1, s = cnt % NS;
                const uint32_t buf = (g + y) & 1;
                alive = warp_wait(&sh->full[s], (cnt / NS) & 1, abort_flag, p.dev_status);
                if (!alive) break;
                const uint32_t phase = ((g + y) >> 1) & 1;
                if (tiles.keys.masked(p, tiles.base(y))) {
                    alive = warp_wait<true>(&sh->v_clean[vcnt % kInTurn], (vcnt / kInTurn) & 1,
                                            abort_flag, p.dev_status);
                    ++vcnt;
                }
                alive = alive && warp_wait(&sh->p_full[buf], phase, abort_flag, p.dev_status);
                if (!alive) break;
                tc::tc_fence_after();
#pragma unroll
                for (int i = 0; i < kKeys / 16; ++i)
                    tc::mma_bf16_ts_pair(t_o, t_s + buf * kKeys + i * 8,
                                         v_desc + (s * (kStage / 16) + i * 128), id_pv,
                                         y > 0 || i > 0);
                tc::mma_commit_pair(&sh->empty[s]);
                tc::mma_commit_pair(&sh->pv_done[buf]);
                ++cnt;
            }
            g += n;
        }
        if (!alive) {
            tc::mma_commit_pair(&sh->drain);
            tc::mbar_wait(&sh->drain, 0);
        }
    } else if (warp == 2 || warp == 3) {
        // ---------------------------------------------------------------- V of masked tiles
        // What not every row of the pair sees must be finite where it meets a weight of 0:
        // rows of keys that hold something else, and rows behind the last key, are zeroed
        // while the softmax of the tile runs.
        uint32_t cnt = 0, vcnt = 0;   // stages, masked tiles before this item's
        int turn = 0;
        bool alive = true;
        while (const Job *job = take(alive)) {
            const Job tiles = *job;
            give_back();
            const int n = tiles.n;
            int i = 0;
            for (int x = 0; x < n; ++x) {
                const int t0 = tiles.base(x);
                if (!tiles.keys.masked(p, t0)) continue;
                alive = warp_wait(&sh->v_ready[vcnt % kInTurn], (vcnt / kInTurn) & 1, abort_flag,
                                  p.dev_status);
                if (!alive) break;
                ++vcnt;
                if (warp == 2 && i == 0) {   // the record of the item after the next
                    const int after = turn + 2 < kRecords ? turn + 2 : turn + 2 - kRecords;
                    (&sh->bad[after][0][0])[lane] = 0;
                    if (lane == 0) sh->poison[after] = 0;
                }
                // stages in order: K(0), K(1) V(0), K(2) V(1), ..., V(n - 1)
                const uint32_t stage = (cnt + (x + 1 < n ? x + 2 : n) * KST + x) % NS;
                // this warp's keys 64 (warp - 2) + lane and 32 further on, both at once
                const int key = (warp - 2) * 64 + lane;
                uint8_t *v_row = smem + stage * kStage + key * 128;
                const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
                __nv_bfloat162 acc[2][4];
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e / 4][e % 4] = zero;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(
                        v_row + (e & 1) * 4096 + (e >> 4) * 16384 + (((e >> 1) + key) & 7) * 16);
                    const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        acc[e & 1][q] = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&word[q]),
                                                zero, acc[e & 1][q]);
                }
                bool wrote = false;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const bool stale = t0 + key + w * 32 > tiles.keys.hi;
                    const __nv_bfloat162 all = __hadd2(__hadd2(acc[w][0], acc[w][1]),
                                                       __hadd2(acc[w][2], acc[w][3]));
                    const bool bad = !stale && (__hisnan(all.x) || __hisnan(all.y));
                    if (bad || stale) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            *reinterpret_cast<uint4 *>(v_row + w * 4096 + (e >> 3) * 16384 +
                                                       (e & 7) * 16) = make_uint4(0, 0, 0, 0);
                        tc::fence_proxy_async_smem();
                    }
                    const uint32_t mask = __ballot_sync(kFull, bad);
                    wrote |= __any_sync(kFull, bad || stale) != 0;
                    if (mask && lane == 0) {
                        for (int r = 0; r < 2; ++r) {
                            tc::or_cluster_u32(
                                tc::map_to_rank(&sh->bad[turn][i][(warp - 2) * 2 + w], r), mask);
                            tc::or_cluster_u32(tc::map_to_rank(&sh->poison[turn], r), 1);
                        }
                    }
                }
                ++i;
                __syncwarp();
                if (lane == 0) {
                    const uint32_t bar = tc::map_to_rank(&sh->v_clean[(vcnt - 1) % kInTurn], 0);
                    if (wrote)
                        tc::mbar_arrive_cluster(bar);
                    else
                        tc::mbar_arrive_remote(bar);
                }
            }
            cnt += n * (KST + 1);
            if (i > 0) turn = turn == kRecords - 1 ? 0 : turn + 1;
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- softmax
        const int part = (warp - 4) / 4, quad = warp % 4;   // keys 64 part .. of a tile; lanes
        const int row = quad * 32 + lane;                   // TMEM lane
        const uint32_t lanes = (uint32_t)quad << 21;
        const int token = row / p.group, head = row - token * p.group;
        const int inv_group = 65536 / p.group + 1;   // r inv_group >> 16 = r / group, r < 128
        // The sign of the scale is in the product's descriptor.  0 would turn the -inf of a masked
        // score into NaN: the least number above it takes every finite score below 2^-20.
        const float scale = fmaxf(fabsf(p.scale_log2), FLT_TRUE_MIN);
        uint32_t g = 0;   // tiles before this item's
        int turn = 0;     // which of the poison records
        int told = 0;     // whose place is whose
        bool alive = true;
        while (const Job *job = take(alive)) {
            const Job &tiles = *job;   // given back when the output's places are known
            const int n = tiles.n, lo_row = tiles.it.j0 + rank * plan.tokens;
            const int pos = tiles.it.ctx + min(lo_row + token, tiles.it.n - 1);
            float m = -INFINITY, l = 0.f;
            bool has_masked = false, large = false, rounded = false;
            for (int x = 0; x < n; ++x) {
                const uint32_t buf = (g + x) & 1;
                alive = alive && warp_wait(&sh->s_full[buf], ((g + x) >> 1) & 1, abort_flag,
                                           p.dev_status);
                tc::tc_fence_after();
                const uint32_t t_x = t_s + buf * kKeys + lanes;
                uint32_t s[64];
                tc::tmem_ld32(t_x + part * 64, s);
                tc::tmem_ld32(t_x + part * 64 + 32, s + 32);
                tc::tmem_ld_wait();
                const int t0 = tiles.base(x);
                if (tiles.keys.masked(p, t0)) {
                    has_masked = true;
                    const int first = t0 + part * 64;
                    uint64_t see = low_bits(pos - first + 1);
                    if (p.window > 0)
                        see &= ~low_bits(pos - p.window + 1 - first) | low_bits(p.sinks - first);
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        if (!((i < 32 ? (uint32_t)see >> i : (uint32_t)(see >> 32) >> (i - 32)) & 1u))
                            s[i] = 0xff800000u;
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 64; ++i) top[i & 3] = fmaxf(top[i & 3], __uint_as_float(s[i]));
                const float own = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                // After this barrier both threads of a row hold their scores, so the weights
                // may take their place.
                sh->row[part ^ told][row] = own;
                if (rows_barrier(quad, !alive)) {
                    alive = false;
                    break;
                }
                told ^= 1;
                const float tm = fmaxf(own, sh->row[part ^ told][row]) * scale;
                const bool grow = tm > m + kSlack;
                if (__any_sync(kFull, grow)) {
                    const float m_new = grow ? tm : m;
                    const float f = m == m_new ? 1.f : fast_exp2(m - m_new);
                    m = m_new;
                    l *= f;
                    // (rows of no query hold anything, and no row changes another's bits)
                    large = fabsf(m) >= kRounded && fabsf(m) < INFINITY &&
                            token < min(plan.tokens, tiles.it.n - lo_row);
                    rounded = __any_sync(kFull, large);
                    if (x > 0) {
                        // each of the two warps scales half of the columns
                        alive = warp_wait(&sh->pv_done[buf ^ 1], ((g + x - 1) >> 1) & 1, abort_flag,
                                          p.dev_status);
                        tc::tc_fence_after();
#pragma unroll 1
                        for (int i = part * (kDV / 2); i < (part + 1) * (kDV / 2); i += 32) {
                            uint32_t o[32];
                            tc::tmem_ld32(t_o + lanes + i, o);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tc::tmem_st32(t_o + lanes + i, o);
                        }
                        tc::tmem_st_wait();
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                auto weigh = [&](int i, float a, float d) {
                    const uint32_t w = pack_bf16(fast_exp2(a), fast_exp2(d));
                    s[i / 2] = w;
                    sum[i / 2 & 3] += bf16lo(w) + bf16hi(w);
                };
                if (rounded) {
                    auto less = [&](uint32_t score) {
                        const float x = __uint_as_float(score);
                        return large ? __fsub_rn(__fmul_rn(x, scale), ref) : fmaf(x, scale, -ref);
                    };
#pragma unroll
                    for (int i = 0; i < 64; i += 2) weigh(i, less(s[i]), less(s[i + 1]));
                } else {
#pragma unroll
                    for (int i = 0; i < 64; i += 2)
                        weigh(i, fmaf(__uint_as_float(s[i]), scale, -ref),
                              fmaf(__uint_as_float(s[i + 1]), scale, -ref));
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tc::tmem_st32(t_x + part * 32, s);
                tc::tmem_st_wait();
                tc::tc_fence_before();
                __syncwarp();
                if (alive && lane == 0)
                    tc::mbar_arrive_remote(tc::map_to_rank(&sh->p_full[buf], 0));
            }
            if (!alive) break;
            g += n;
            // While the last product runs: a row's sum, its place.
            sh->row[part ^ told][row] = l;
            if (rows_barrier(quad, !alive)) {
                alive = false;
                break;
            }
            told ^= 1;
            l += sh->row[part ^ told][row];
            const bool partial = tiles.it.splits > 1;
            const int split = tiles.it.split, d0 = tiles.it.vh * kDV;
            const int held = min(plan.tokens, tiles.it.n - lo_row);   // tokens that have rows here
            const size_t at = ((size_t)tiles.it.b * p.k + lo_row) * p.q_heads +
                              tiles.it.c * p.group;
            if (partial && token < held && d0 == 0 && part == 0)
                plan.part_ml[(at + token * p.q_heads + head) * plan.splits + split] =
                    make_float2(m, l);
            float f = partial ? 1.f : 1.f / l;
            // where this thread writes of the warp's rows 4 e + lane / 8 (null: no such row)
            const size_t row_bytes = partial ? (size_t)plan.splits * D * 4 : (size_t)D * 2;
            uint8_t *const whole = partial ? reinterpret_cast<uint8_t *>(
                                                 plan.part_o + (size_t)split * D + d0)
                                           : reinterpret_cast<uint8_t *>(p.out + d0);
            uint8_t *to[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int rr = quad * 32 + e * 4 + lane / 8, tt = rr * inv_group >> 16;
                to[e] = tt < held ? whole + (at + tt * p.q_heads + rr - tt * p.group) * row_bytes +
                                        (lane & 7) * 16
                                  : nullptr;
            }
            // The last scores say that the product two tiles before is done, no more: with one
            // barrier for all products this wait could meet a phase too early or too late.
            alive = warp_wait<true>(&sh->pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag,
                                    p.dev_status);
            if (!alive) break;
            tc::tc_fence_after();
            bool poisoned = false;
            if (has_masked && *(volatile uint32_t *)&sh->poison[turn]) {
                for (int x = 0, i = 0; x < n; ++x) {
                    const int t0 = tiles.base(x);
                    if (!tiles.keys.masked(p, t0)) continue;
                    for (int w = 0; w < 4; ++w)
                        for (uint32_t bits = sh->bad[turn][i][w]; bits; bits &= bits - 1) {
                            const int t = t0 + w * 32 + __ffs(bits) - 1;
                            poisoned |=
                                t <= pos && (p.window == 0 || t > pos - p.window || t < p.sinks);
                        }
                    ++i;
                }
            }
            if (has_masked) turn = turn == kRecords - 1 ? 0 : turn + 1;
            if (poisoned) f = NAN;
            give_back();
            // O leaves through shared memory, 128 bytes of each of the warp's 32 rows at a
            // time, so that eight lanes write a whole line.
            uint8_t *s_out = smem + L::kOffOut + (warp - 4) * 4096;
            const uint8_t *s_from = s_out + lane / 8 * 128;
            auto leave = [&](int column_bytes) {
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int r = e * 4 + lane / 8;
                    const uint4 v = *reinterpret_cast<const uint4 *>(s_from + e * 512 +
                                                                     ((lane ^ r) & 7) * 16);
                    if (to[e]) *reinterpret_cast<uint4 *>(to[e] + column_bytes) = v;
                }
                __syncwarp();
            };
#pragma unroll 1
            for (int i = part * (kDV / 2); i < (part + 1) * (kDV / 2); i += 32) {
                uint32_t o[32];
                tc::tmem_ld32(t_o + lanes + i, o);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                if (partial) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<uint4 *>(s_out + lane * 128 + ((e ^ lane) & 7) * 16) =
                            make_uint4(o[e * 4], o[e * 4 + 1], o[e * 4 + 2], o[e * 4 + 3]);
                    leave(i * 4);
                    continue;
                }
                const int half = (i & 32) / 8;   // of the 128 bytes
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t w[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        w[z] = pack_bf16(__uint_as_float(o[e * 8 + 2 * z]),
                                         __uint_as_float(o[e * 8 + 2 * z + 1]));
                    *reinterpret_cast<uint4 *>(
                        s_out + lane * 128 + (((e + half) ^ lane) & 7) * 16) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (half) leave((i - 32) * 2);
            }
            if constexpr (L::kOutInQ) {
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sh->q_empty);
            }
            tc::tc_fence_before();
        }
        // Requests rejected on the device, by the pair that has the first pair's work
        // (it may have been taken over).
        const bool rejects = alive && sh->job[(taken - 1) % kJobs].it.b != 0;
        for (int first = 0; rejects && first < p.batch; first += 32) {
            const int mine = first + lane;
            uint32_t bad = __ballot_sync(
                kFull, mine < p.batch && !request_ok(p, load_request(p, mine)));
            for (; bad; bad &= bad - 1) {
                if (threadIdx.x == 128) set_status(p.dev_status, CARAT_DEV_BAD_CONTEXT);
                const size_t rows = (size_t)p.k * p.q_heads;
                uint4 *o = reinterpret_cast<uint4 *>(p.out + (first + __ffs(bad) - 1) * rows * D);
                for (size_t i = rank * kSoftmax + threadIdx.x - 128; i < rows * (D / 8);
                     i += 2 * kSoftmax)
                    o[i] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_arrive();
    tc::cluster_wait();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc_pair(tmem, 512);
    }
}

// Merges the pieces of split items: 16 bytes of a row of the output a thread, kFlight
// pieces' loads in flight.  With one row a CTA the first of them are on their way before it
// is known how many pieces there are (one latency, not three after one another).  Rows for
// more CTAs than run at once (MANY) are shared out, `per` for each, and those of requests in
// one piece passed over without a load: a CTA for each of 64000 that needed none took 70 us.
template <int D, bool MANY>
__global__ void __launch_bounds__(D / 4) paged_chunk_merge_kernel(
    const __grid_constant__ PagedChunkParams p, const Plan plan, int rows, int per) {
    constexpr int kFlight = 8;
    wait_for_prior_launch();
    let_next_launch_start();
    const int last = MANY ? min(rows, (int)(blockIdx.x + 1) * per) : blockIdx.x + 1;
    float2 l[kFlight];
    float4 v[kFlight];
    for (int at = MANY ? blockIdx.x * per : blockIdx.x; at < last;) {
        const int token = at / p.q_heads;
        const int b = token / p.k, j = token - b * p.k;
        const float2 *ml = plan.part_ml + (size_t)at * plan.splits;
        const float4 *o = reinterpret_cast<const float4 *>(plan.part_o +
                                                           (size_t)at * plan.splits * D) +
                          threadIdx.x;
        auto load = [&](int s0) {
#pragma unroll
            for (int i = 0; i < kFlight; ++i)
                if (s0 + i < plan.splits) {
                    l[i] = ml[s0 + i];
                    v[i] = o[(size_t)(s0 + i) * (D / 4)];
                }
        };
        if (!MANY) load(0);
        const Request rq = load_request(p, b);
        const int pieces = plan.pieces[b];
        bool skip = !request_ok(p, rq) || j >= rq.n;
        // A number that the attention did not write this time (it stopped on a timeout before
        // the request) is not used: it may stand for more pieces than there are places.
        if (!skip && (pieces < 1 || pieces > plan.splits)) {
            if (threadIdx.x == 0) set_status(p.dev_status, CARAT_DEV_TIMEOUT);
            skip = true;
        }
        if (skip || pieces == 1) {   // (one piece: written whole)
            if (!MANY) return;
            at = (b + 1) * p.k * p.q_heads;
            continue;
        }
        if (MANY) load(0);
        const int j0 = j / (2 * plan.tokens) * 2 * plan.tokens;
        const Keys keys(p, (int)rq.ctx + j0, (int)rq.ctx + min(j0 + 2 * plan.tokens, rq.n) - 1);
        float top = -INFINITY, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        int from = 0;
#pragma unroll 1
        for (int s0 = 0; s0 < pieces; s0 += kFlight) {
            if (s0 > 0) load(s0);
            float most = top;
            bool have[kFlight];   // pieces without a tile wrote nothing
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const int to = split_at(keys.count, s0 + i + 1, pieces);
                have[i] = s0 + i < pieces && to > from;
                from = to;
                if (have[i]) most = fmaxf(most, l[i].x);
            }
            const float ref = most == -INFINITY ? 0.f : most;
            const float keep = fast_exp2(top - ref);
            top = most;
            sum *= keep;
            acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                if (!have[i]) continue;
                const float w = fast_exp2(l[i].x - ref);
                sum = fmaf(w, l[i].y, sum);
                acc.x = fmaf(w, v[i].x, acc.x);
                acc.y = fmaf(w, v[i].y, acc.y);
                acc.z = fmaf(w, v[i].z, acc.z);
                acc.w = fmaf(w, v[i].w, acc.w);
            }
        }
        const float f = 1.f / sum;
        reinterpret_cast<uint2 *>(p.out + (size_t)at * D)[threadIdx.x] =
            make_uint2(pack_bf16(acc.x * f, acc.y * f), pack_bf16(acc.z * f, acc.w * f));
        if (!MANY) return;
        ++at;
    }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// What pieces may leave, where the items are few (kFewItems for each pair) and where not.
constexpr size_t kPieceBytes = (size_t)128 << 20, kPieceBytesMany = (size_t)32 << 20;
constexpr int kFewItems = 3;

struct Sizes {
    Plan plan;
    size_t ml, o, total;
};

// The most key tiles that `tokens` tokens one after another can see.
long long tiles_most(int tokens, int window, int sinks, int capacity) {
    const long long all = capacity / kKeys;
    if (window == 0) return all;
    return std::min(all, ((long long)window + tokens) / kKeys + 2 +
                             ((long long)sinks + kKeys - 1) / kKeys);
}

// For a page table of `capacity` keys; the workspace is that of any (INT_MAX), without a window.
Sizes sizes_of(int batch, int k, int q_heads, int kv_heads, int head_dim, int window, int sinks,
               int capacity) {
    Sizes z{};
    z.plan.tokens = kRows / (q_heads / kv_heads);
    z.plan.halves = head_dim / kDV;
    const int tiles = (k + 2 * z.plan.tokens - 1) / (2 * z.plan.tokens);
    const long long items = (long long)batch * kv_heads * tiles * z.plan.halves;
    const int pairs = device_sm_count() / 2;
    const size_t row = (size_t)batch * k * q_heads * head_dim * sizeof(float);
    // Few items: as many pieces as make one for every pair.  Several requests without a window
    // may differ much in length: up to kUnits pieces a pair, within what may be left.  Planning
    // and an extra launch cost 3 us and more, and pieces are not taken over; one long request
    // among short ones costs up to half of the call.  us, without and with pieces, requests of
    // 64 tokens behind 500 to 30000 (16/2 heads of 512, 128 items) 575 and 315, 3 of 512 behind
    // 500 to 12000 (192 items) 366 and 241, 5 of 842 behind up to 11349 (70 items) 113 and 71;
    // but 8 of up to 512 behind up to 8000 (16/8 of 256, 256 items, 64 MB) 45 and 67.
    // An item has no more pieces than its window and the page table can have key tiles, and
    // few tiles are not split at all, as a merge costs kMergeCost of them.  us, before and
    // with that: 5 tokens in a table of 384 keys (5/1 heads of 256) 21 and 11, 21 tokens under
    // a window of 1024 (10/2) 18.7 and 14.2, 31 prompts of up to 283 (4/2) 27.5 and 21.7.
    const long long most_tiles = tiles_most(2 * z.plan.tokens, window, sinks, capacity);
    const long long one = items > 0 && most_tiles > kMergeCost
                              ? std::max<long long>(1, std::min(pairs / items, most_tiles))
                              : 1;
    z.plan.splits = (int)one;
    if (items > 0 && items <= (long long)kUnits / 2 * pairs && batch > 1 && window == 0 &&
        most_tiles > kPieceCost + kMergeCost) {
        const long long most = std::min({kUnits * pairs / items, (long long)pairs, most_tiles});
        const size_t room = items <= kFewItems * (long long)pairs ? kPieceBytes : kPieceBytesMany;
        z.plan.splits = (int)std::max(one, std::min<long long>(most, room / row));
        z.plan.by_length = z.plan.splits > 1;
    }
    // Split items: every pair of the grid runs at once.  Else a pair that finds no item costs
    // about a microsecond (a padded batch has many): the grid is at most kUnits times the
    // pairs that run at once.
    z.plan.units = (int)std::min<long long>(
        items * z.plan.splits, (z.plan.splits > 1 ? 1LL : (long long)kUnits) * pairs);
    if (z.plan.splits > 1) {
        const size_t rows = (size_t)batch * k * q_heads * z.plan.splits;
        z.ml = align256(rows * sizeof(float2));
        z.o = align256(rows * head_dim * sizeof(float));
        z.total = z.ml + z.o + align256((size_t)batch * sizeof(int));
    }
    return z;
}

template <int D>
cudaError_t launch(const PagedChunkParams &p, Sizes &z, cudaStream_t stream) {
    using L = Lay<D>;
    char *w = static_cast<char *>(p.workspace);
    z.plan.part_ml = reinterpret_cast<float2 *>(w);
    z.plan.part_o = reinterpret_cast<float *>(w + z.ml);
    z.plan.pieces = reinterpret_cast<int *>(w + z.ml + z.o);
    CUtensorMap map_q{}, map_k{}, map_v{};
    const uint64_t row = (uint64_t)p.kv_heads * D * 2;
    const uint64_t dims[4] = {64, (uint64_t)p.num_pages * p.page_rows, D / 64, (uint64_t)p.kv_heads};
    const uint64_t strides[3] = {row, 128, D * 2};
    const uint32_t box_k[4] = {64, 64, 4, 1}, box_v[4] = {64, kKeys, 2, 1};
    const uint64_t dims_q[4] = {D, (uint64_t)p.q_heads, (uint64_t)p.k, (uint64_t)p.batch};
    const uint64_t strides_q[3] = {D * 2, (uint64_t)p.q_heads * D * 2,
                                   (uint64_t)p.k * p.q_heads * D * 2};
    const uint32_t box_q[4] = {64, (uint32_t)p.group, (uint32_t)z.plan.tokens, 1};
    if (!make_bf16_tensor_map(&map_q, p.q, 4, dims_q, strides_q, box_q, true) ||
        !make_bf16_tensor_map(&map_k, p.k_pages, 4, dims, strides, box_k, true) ||
        !make_bf16_tensor_map(&map_v, p.v_pages, 4, dims, strides, box_v, true))
        return cudaErrorInvalidValue;
    auto kernel = paged_chunk_kernel<D>;
    static std::atomic<int> configured[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev].store(1, std::memory_order_release);
    }
    e = launch_dependent(kernel, dim3(2 * z.plan.units), dim3(kThreads),
                         L::kAlloc, stream, p, z.plan, map_q, map_k, map_v);
    if (e != cudaSuccess || z.plan.splits == 1) return e;
    const int rows = p.batch * p.k * p.q_heads;
    const int at_once = device_sm_count() * (2048 / (D / 4)), per = (rows - 1) / at_once + 1;
    return launch_dependent(per > 1 ? paged_chunk_merge_kernel<D, true>
                                    : paged_chunk_merge_kernel<D, false>,
                            dim3((rows - 1) / per + 1), dim3(D / 4), 0, stream, p, z.plan, rows,
                            per);
}

}  // namespace

// Few rows of many requests at head_dim 512: the stream-K kernel with keys as the products'
// long side (attention_tc.cuh), where a CTA pair would spend 256 rows' products on a
// request's few, twice over for the scores.  It takes 25 us for little or no work, so the
// requests have to be able to fill kStepTiles key tiles of KV heads.  Measured, us, pairs
// against it: 64 requests of 2 KV heads and 4 tokens under a window of 4096 (4480 tiles) 208
// and 157, of 1024 (1280) 94 and 90, of up to 1000 keys (1024) 73 and 63, 64 of one token and
// up to 16000 keys 417 and 210, 8 of 4 tokens and up to 32768 keys (4096) 100 and 81; but 32
// under a window of 1024 (640) 52 and 58, 16 under it (288) 28 and 39, 16 of up to 1000 keys
// (256) 29 and 37, and 4 of 6005 keys 37 and 42.
constexpr int kStepUnits = 16, kStepTiles = 640;

static bool few_rows(int batch, int k, int q_heads, int kv_heads, int head_dim, int window,
                     int sinks, int capacity) {
    const long long units = batch * (long long)kv_heads;
    return units >= kStepUnits && tc_window_supported(head_dim, q_heads / kv_heads, k) &&
           units * tiles_most(k, window, sinks, capacity) > kStepTiles;
}

struct StepSizes {
    int grid;
    size_t ml, o, total;
};

static StepSizes step_sizes(int batch, int k, int q_heads, int kv_heads, int head_dim) {
    const int n = tc_rows_per_tile(q_heads / kv_heads, k);
    StepSizes z{};
    z.grid = tc_ctas_per_sm(head_dim, n, false) * device_sm_count();
    const size_t slots = (size_t)z.grid * 2 * n;
    z.ml = align256(slots * sizeof(float2));
    z.o = align256(slots * (size_t)head_dim * sizeof(float));
    z.total = z.ml + z.o + align256((size_t)batch * kv_heads * sizeof(int4));
    return z;
}

static cudaError_t launch_step(const PagedChunkParams &p, cudaStream_t stream) {
    const StepSizes z = step_sizes(p.batch, p.k, p.q_heads, p.kv_heads, p.head_dim);
    char *w = static_cast<char *>(p.workspace);
    AttnParams a{};
    a.q = p.q;
    a.k_base = p.k_pages;
    a.v_base = p.v_pages;
    a.context_lengths = p.context_lengths;
    a.new_counts = p.new_counts;
    a.out16 = p.out;
    a.part_ml = reinterpret_cast<float2 *>(w);
    a.part_o = reinterpret_cast<float *>(w + z.ml);
    a.units = reinterpret_cast<int4 *>(w + z.ml + z.o);
    a.dev_status = p.dev_status;
    a.batch = p.batch;
    a.k = p.k;
    a.q_heads = p.q_heads;
    a.kv_heads = p.kv_heads;
    a.head_dim = p.head_dim;
    a.group = p.group;
    a.rows = p.group * p.k;
    a.window = p.window;
    a.sinks = p.window > 0 ? p.sinks : 0;
    a.capacity = p.capacity;
    a.page_table = p.page_table;
    a.max_pages = p.max_pages;
    a.page_rows = p.page_rows;
    a.num_pages = p.num_pages;
    a.scale_log2 = p.scale_log2;
    a.source = KeySource::kPagedWindow;
    return launch_attention_tc_window(a, z.grid, stream);
}

bool paged_chunk_supported(int head_dim) { return head_dim == 256 || head_dim == 512; }

size_t paged_chunk_workspace(int batch, int k, int q_heads, int kv_heads, int head_dim) {
    const size_t pairs = sizes_of(batch, k, q_heads, kv_heads, head_dim, 0, 0, INT_MAX).total;
    const size_t step = few_rows(batch, k, q_heads, kv_heads, head_dim, 0, 0, INT_MAX)
                            ? step_sizes(batch, k, q_heads, kv_heads, head_dim).total
                            : 0;
    return std::max(pairs, step);
}

cudaError_t launch_paged_chunk_attention(const PagedChunkParams &p, cudaStream_t stream) {
    if (few_rows(p.batch, p.k, p.q_heads, p.kv_heads, p.head_dim, p.window, p.sinks, p.capacity))
        return launch_step(p, stream);
    Sizes z = sizes_of(p.batch, p.k, p.q_heads, p.kv_heads, p.head_dim, p.window, p.sinks,
                       p.capacity);
    return p.head_dim == 256 ? launch<256>(p, z, stream) : launch<512>(p, z, stream);
}

}  // namespace carat
