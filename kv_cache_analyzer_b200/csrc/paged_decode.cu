// paged_decode.cu -- paged attention of few rows per sequence (single tokens
// above all): at most 32 packed rows, (query row, head of the group), per
// sequence and K/V head.  Same formula and layout as paged_attention.cu.
//
// Bound by the cache's bytes, so the design serves one thing: K/V tiles in
// flight on every SM until the last byte.  One persistent CTA per SM takes an
// equal share of all key tiles, counted through sequences, heads and keys in
// that order, whatever the lengths (or, for few sequences, a part of one of
// them: item_quota); where a share begins or ends inside a
// sequence's head, the CTA leaves a partial (O, m, l) and a second kernel, its
// programmatic dependent, adds the parts in order.  Within a CTA the loads of
// the next (sequence, head) start while the last one is still being worked
// on: all barriers count through, and Q has two buffers.
//
// 128 KB of K/V tiles per SM: with 96 KB one token each of 32 sequences
// (d = 128, 2.8 GB of K/V) took 471 us, with 128 or 160 KB 405, with 192 KB
// 434, as the SMs then finish further apart (340 to 435 us).
//
// Reading 7 TB/s takes the card to its power limit by itself, so the tensor
// core's share of the power costs time, though its time does not: the MMAs
// have the smallest M that holds the rows (64 for 16 packed rows, 128 for 32),
// and their other rows are zeros, kept around Q.  The same 32 sequences over
// and over, at 1000 W: 480 us with M = 128 over whatever lay behind Q (SM clock
// 1,080 MHz), 448 with zeros there (1,300), 424 with M = 64 (1,540); a plain
// sum of as many bytes takes 408 (1,680).  After a pause, 405 us: 6.9 TB/s.
//
// P is rounded to BF16 for P V as in paged_attention.cu.  Two BF16 terms of P
// would cost no bytes here, but one more MMA a tile (the power counts, above),
// and a row's precision would depend on the form that its call takes.
//
// 7 warps:  0, 1  softmax of streams 0 and 1 (even and odd key tiles; thread =
// packed row.  Stream 1's operand starts R rows before Q, so its rows fall
// into the TMEM lanes that warp 1 reaches, on another scheduler; with M = 64
// every quarter of the lanes holds 16 rows), 2 MMA issuer, 3 clears V rows past
// the visible length, 4 planner: it walks the device's lists once and hands
// the CTA's segments (runs of key tiles of one sequence and head) to the
// others through a small ring, 5 producer of Q and K, 6 producer of V.  The
// two streams' parts are joined through shared memory at the end of each
// segment.
//
// A segment of one or two tiles costs 4.7 us whatever it reads (2,048 sequences
// of 128 tokens: 515 us); the MMAs of one segment start when those of the last
// are issued.  Letting them run on into the next made that 323 us, and long
// sequences of d = 64 4.5% slower.
//
// Every wait is bounded (those that span a segment by the longest one's tiles).
// The partial slots of a CTA are marked missing before it starts, so that rows
// of a CTA that gave up are not written.
#include "paged_tile.cuh"

namespace jano {
namespace {

constexpr int kThreads = 224;                // two warps per scheduler at most: 255 registers for a thread's S row
constexpr int kMaxRows = 32;                 // packed rows at most
constexpr int kSegs = 4;                     // segments in the planner's ring

// A run of key tiles of one (sequence, K/V head).
struct Seg {
    int row0, rows;      // query rows
    int seq, head;
    int seen;            // keys that any of the rows sees
    int kt0, n;          // first key tile, key tiles (0: no more segments)
    int part;            // partial slot of the CTA that it goes to; -1: the whole item, straight to out
};

// R: packed rows of the form (16 or 32), a quarter of its MMAs' M.
template <int HD, int R>
struct Layout {
    static constexpr int kM = 4 * R;
    static constexpr int kPanels = HD / 64;
    static constexpr uint32_t kTile = kPanels * kPanel;
    static constexpr uint32_t kQRows = R * 128;                   // bytes of the R rows of one 64-column panel
    static constexpr uint32_t kQPanel = kM * 128;                 // ... and of the zeros that follow
    static constexpr uint32_t kQ = kPanels * kQPanel;             // one Q buffer
    // stream 1's O, float [R][kStageRow] (padded: adjacent rows on different
    // banks), its (m, l), then R rows of zeros (stream 1's operand starts
    // there) and the two Q buffers
    static constexpr uint32_t kStageRow = HD + 4;
    static constexpr uint32_t kStageMl = R * kStageRow * 4;
    static constexpr uint32_t kZeros = (kStageMl + 32 * 8 + 1023) / 1024 * 1024;
    static constexpr uint32_t kQ0 = kZeros + kQRows;
    static constexpr uint32_t kRingK = kQ0 + 2 * kQ;
    static constexpr int kSlots = 128 * 1024 / kTile / 2;         // K tiles, and V tiles, see above
    static constexpr uint32_t kRingV = kRingK + kSlots * kTile;
    static constexpr uint32_t kBar = kRingV + kSlots * kTile;
    static constexpr int bFullK = 0;                   // [kSlots]
    static constexpr int bEmptyK = bFullK + kSlots;    // [kSlots]
    static constexpr int bFullV = bEmptyK + kSlots;    // [kSlots] landed and cleared past the last key
    static constexpr int bEmptyV = bFullV + kSlots;    // [kSlots]
    static constexpr int bLand = bEmptyV + kSlots;     // [kSlots] a ragged V tile landed, not yet cleared
    static constexpr int bQFull = bLand + kSlots;      // [2]
    static constexpr int bQEmpty = bQFull + 2;         // [2]
    static constexpr int bSFull = bQEmpty + 2;         // [2]
    static constexpr int bPHalf = bSFull + 2;          // [2]
    static constexpr int bPFull = bPHalf + 2;          // [2]
    static constexpr int bOFull = bPFull + 2;          // [2]
    static constexpr int bOEmpty = bOFull + 2;         // [2]
    static constexpr int bStage = bOEmpty + 2;
    static constexpr int bStageFree = bStage + 1;
    static constexpr int bZeros = bStageFree + 1;      // the rows around Q are cleared
    static constexpr int bSegFull = bZeros + 1;        // [kSegs]
    static constexpr int bSegEmpty = bSegFull + kSegs; // [kSegs]
    static constexpr int bFinal = bSegEmpty + kSegs;
    static constexpr int kNumBars = bFinal + 1;
    static constexpr uint32_t kSeg = kBar + 8 * kNumBars;         // Seg [kSegs]
    static constexpr uint32_t kMisc = kSeg + kSegs * (uint32_t)sizeof(Seg);
    static constexpr uint32_t kBytes = kMisc + 16;                // tmem base, abort flag, share is empty
    static constexpr uint32_t kAlloc = kBytes + 1024;             // slack for 1 KB alignment
    static_assert(kAlloc <= 227 * 1024, "shared memory budget");
    static_assert(kQ0 % 1024 == 0 && kRingK % 1024 == 0 && kBar % 8 == 0, "alignment");
};

struct Args {
    const int32_t* table;
    const int32_t* lens;
    const int32_t* cu;
    const int32_t* limits;
    int n_seqs, max_pages, n_pages, page_shift;
    int n_rows, max_rows, max_len;
    int kv_heads, group, tile_rows;    // query heads per K/V head, query rows per tile
    float scale_log2;
    __nv_bfloat16* out;
    long long out_ld;
    float* part_o;                     // [2 * CTAs][part_rows][d]
    float2* part_ml;                   // [2 * CTAs][part_rows]
    int part_rows;
    int* err;
};

// One sequence as this lane sees it: its rows, the keys they see, key tiles
// per head (one, all masked, for rows that see nothing: they are written too).
struct SeqInfo {
    int row0, rows, seen, tiles;
};
__device__ __forceinline__ SeqInfo seq_info(const Args& a, int s, bool report) {
    SeqInfo q{0, 0, 0, 0};
    if (s >= a.n_seqs) return q;
    const int lo = __ldg(a.cu + s), hi = __ldg(a.cu + s + 1), len = __ldg(a.lens + s);
    const bool ok = lo >= 0 && lo <= hi && hi <= a.n_rows && hi - lo <= a.max_rows && len >= 0 && len <= a.max_len &&
                    (s > 0 || lo == 0);
    if (!ok && report) raise_error(a.err, JANO_EINDEX);
    if (!ok || hi == lo) return q;
    q.row0 = lo;
    q.rows = hi - lo;
    q.seen = len;
    if (a.limits) {
        int most = 0;
        for (int r = lo; r < hi; ++r) most = max(most, __ldg(a.limits + r));
        q.seen = min(len, most);
    }
    q.tiles = max(1, (q.seen + BN - 1) / BN);
    return q;
}
// A row of O from TMEM, all columns in one round trip.
template <int HD>
__device__ __forceinline__ void load_row(uint32_t tO, uint32_t (&o)[HD]) {
#pragma unroll
    for (int c = 0; c < HD / 32; ++c) ptx::tmem_ld32(tO + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&o[32 * c]));
    ptx::tmem_wait_ld();
}
__device__ __forceinline__ int warp_sum_to(int v) {    // inclusive prefix sum over the lanes
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}
// Equal shares of the tiles, the first `more` ones a tile longer; no more
// shares than give each of them two tiles.
struct Shares {
    int n, each, more;
    __device__ Shares(int total, int ctas) : n(max(1, min((total + 1) / 2, ctas))), each(total / n), more(total - each * n) {}
    __device__ int begin(int c) const { return c * each + min(c, more); }
    __device__ int owner(int tile) const {         // the share that a tile lies in
        const int long_ones = more * (each + 1);
        return tile < long_ones ? tile / (each + 1) : more + (tile - long_ones) / each;
    }
};

// Shares that end with their (sequence, head): each is one of the parts of
// some `quota` tiles that its item is cut into.  Taken where it costs at most
// two tiles more than equal shares of everything: a CTA that goes on to a second
// item drains and fills its pipeline in between, as long as three tiles take
// (one token of 24 heads over 4,096 tokens: the CTAs that cross ended after 15
// to 17 us, the others after 12 to 14; 21.3 us in all, 19.3 without crossing).
// Parts of an item of `tiles`: tiles / quota, rounded up.  The float quotient
// (what this computes counts: integer divisions cost 1 us of start) is only an
// estimate, off by one at most up to 2^19 tiles; what is left over corrects it,
// so that the attention and the merge kernel cut an item alike however each is
// compiled.
__device__ __forceinline__ int item_parts(int tiles, int quota) {
    const int q = (int)__fdividef((float)tiles, (float)quota);
    const int left = tiles - q * quota;
    return q + (left > 0) + (left > quota) - (left <= -quota);
}
// The quota, 0 for equal shares.  The whole warp; n_seqs <= 32, `tiles` the lane's sequence's.
__device__ __forceinline__ int item_quota(const Args& a, int tiles, const Shares& sh, int ctas) {
    const int least = max(2, sh.each + (sh.more > 0));
    int quota = 0;
#pragma unroll 1
    for (int t = least + 2; t >= least && a.n_seqs <= 32; --t) {   // most often the first is one too many
        if (__reduce_add_sync(0xFFFFFFFFu, item_parts(tiles, t)) * a.kv_heads > ctas) break;
        quota = t;
    }
    return quota;
}
// Share c of those: its sequence (a lane), head, part of how many; the item's first share.
struct ItemPart {
    int lane, head, part, parts, first;
    __device__ __forceinline__ ItemPart(const Args& a, int tiles, int quota, int c) {
        const int mine = item_parts(tiles, quota);
        const int upto = warp_sum_to(mine), from = (upto - mine) * a.kv_heads;
        lane = __ffs(__ballot_sync(0xFFFFFFFFu, c >= from && c < from + mine * a.kv_heads)) - 1;
        if (lane < 0) return;                              // no such share
        parts = __shfl_sync(0xFFFFFFFFu, mine, lane);
        const int rem = c - __shfl_sync(0xFFFFFFFFu, from, lane);
        head = rem / parts;
        part = rem - head * parts;
        first = c - part;
    }
};

// The segments of one CTA's share, one after another (a whole warp walks).
struct Walk {
    const Args& a;
    int begin, end;                        // the share, in tiles
    int s0, at;                            // the 32 sequences in hand, and their first tile
    SeqInfo mine;
    int from, upto;                        // this lane's sequence's first tile; tiles of the 32 up to it
    unsigned todo;                         // lanes whose sequences are still to come
    Seg s;
    int tiles, first, item;                // of the sequence in hand; the item's first tile (< end: there is one)
    bool one;                              // the share is s alone (item_quota), not yet handed out

    __device__ __forceinline__ Walk(const Args& args, bool report)
        : a(args), s0(0), at(0), upto(0), todo(0), tiles(0), first(0), item(0), one(false) {
        const int lane = threadIdx.x & 31;
        mine = seq_info(a, lane, report);
        int total = __reduce_add_sync(0xFFFFFFFFu, mine.tiles);
        for (int k = 32; k < a.n_seqs; k += 32)
            total += __reduce_add_sync(0xFFFFFFFFu, seq_info(a, k + lane, report).tiles);
        const Shares sh(total * a.kv_heads, (int)gridDim.x);
        if (const int quota = item_quota(a, mine.tiles, sh, (int)gridDim.x)) {
            begin = end = 0;
            s.head = a.kv_heads;
            const ItemPart it(a, mine.tiles, quota, (int)blockIdx.x);
            if (it.lane < 0) return;
            one = true;
            tiles = __shfl_sync(0xFFFFFFFFu, mine.tiles, it.lane);
            s.row0 = __shfl_sync(0xFFFFFFFFu, mine.row0, it.lane);
            s.rows = __shfl_sync(0xFFFFFFFFu, mine.rows, it.lane);
            s.seen = __shfl_sync(0xFFFFFFFFu, mine.seen, it.lane);
            s.seq = it.lane;
            s.head = it.head;
            const int each = tiles / it.parts, more = tiles - each * it.parts;
            s.kt0 = it.part * each + min(it.part, more);
            s.n = each + (it.part < more);
            s.part = it.parts > 1 ? 0 : -1;
            s0 = 32;
            return;
        }
        begin = end = 0;
        if ((int)blockIdx.x < sh.n) {
            begin = sh.begin(blockIdx.x);
            end = sh.begin(blockIdx.x + 1);
        }
        s.head = a.kv_heads;               // no sequence in hand
        place();
    }
    __device__ __forceinline__ void place() {
        upto = warp_sum_to(mine.tiles);
        from = at + (upto - mine.tiles) * a.kv_heads;
        todo = __ballot_sync(0xFFFFFFFFu, mine.tiles > 0 && from < end && from + mine.tiles * a.kv_heads > begin);
    }
    __device__ __forceinline__ bool next() {
        if (one) {
            one = false;
            return true;
        }
        if (s.head + 1 < a.kv_heads && item + tiles < end) {       // the next head of the sequence in hand
            ++s.head;
            item += tiles;
        } else {
            while (!todo) {
                at += __shfl_sync(0xFFFFFFFFu, upto, 31) * a.kv_heads;
                s0 += 32;
                if (s0 >= a.n_seqs || at >= end) {
                    s.n = 0;
                    return false;
                }
                mine = seq_info(a, s0 + (threadIdx.x & 31), false);
                place();
            }
            const int j = __ffs(todo) - 1;
            todo &= todo - 1;
            tiles = __shfl_sync(0xFFFFFFFFu, mine.tiles, j);
            first = __shfl_sync(0xFFFFFFFFu, from, j);
            s.row0 = __shfl_sync(0xFFFFFFFFu, mine.row0, j);
            s.rows = __shfl_sync(0xFFFFFFFFu, mine.rows, j);
            s.seen = __shfl_sync(0xFFFFFFFFu, mine.seen, j);
            s.seq = s0 + j;
            s.head = begin > first ? (begin - first) / tiles : 0;
            item = first + s.head * tiles;
        }
        const int t0 = max(begin - item, 0), t1 = min(end - item, tiles);
        s.kt0 = t0;
        s.n = t1 - t0;
        s.part = t0 > 0 ? 0 : (t1 < tiles ? 1 : -1);
        return true;
    }
};

template <int HD, int R>
__global__ void __launch_bounds__(kThreads, 1)
paged_decode_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Args a) {
    using L = Layout<HD, R>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    Ctl ctl;
    ctl.bar0 = base + L::kBar;
    ctl.abort = reinterpret_cast<volatile int*>(gbase + L::kMisc + 4);
    ctl.err = a.err;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::kMisc);
    Seg* ring = reinterpret_cast<Seg*>(gbase + L::kSeg);

    if (threadIdx.x == 32) {
        for (int s = 0; s < L::kSlots; ++s) {
            ptx::mbar_init(ctl.bar(L::bFullK + s), 1);
            ptx::mbar_init(ctl.bar(L::bEmptyK + s), 1);
            ptx::mbar_init(ctl.bar(L::bFullV + s), 1);
            ptx::mbar_init(ctl.bar(L::bEmptyV + s), 1);
            ptx::mbar_init(ctl.bar(L::bLand + s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(ctl.bar(L::bQFull + s), 1);
            ptx::mbar_init(ctl.bar(L::bQEmpty + s), 1);
            ptx::mbar_init(ctl.bar(L::bSFull + s), 1);
            ptx::mbar_init(ctl.bar(L::bPHalf + s), 1);
            ptx::mbar_init(ctl.bar(L::bPFull + s), 1);
            ptx::mbar_init(ctl.bar(L::bOFull + s), 1);
            ptx::mbar_init(ctl.bar(L::bOEmpty + s), 1);
        }
        ptx::mbar_init(ctl.bar(L::bStage), 1);
        ptx::mbar_init(ctl.bar(L::bStageFree), 1);
        ptx::mbar_init(ctl.bar(L::bZeros), 3);
        for (int s = 0; s < kSegs; ++s) {
            ptx::mbar_init(ctl.bar(L::bSegFull + s), 1);
            ptx::mbar_init(ctl.bar(L::bSegEmpty + s), 6);   // two producers, MMA, clearing warp, two softmax warps
        }
        ptx::mbar_init(ctl.bar(L::bFinal), 1);
        *ctl.abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 5 && lane == 0) {
        ptx::prefetch_tmap(&tmQ);
        ptx::prefetch_tmap(&tmK);
        ptx::prefetch_tmap(&tmV);
    }
    // Launched before the kernel in front has ended (calls of one token in a row:
    // 19.9 us each, 22.4 without): nothing in global memory is touched before
    // this.  The merge kernel reads the lists as well: it may be launched after.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0 && lane < a.part_rows) {
        // missing until written: a sum of exponentials is never negative
        a.part_ml[(2ll * blockIdx.x) * a.part_rows + lane] = make_float2(-INFINITY, -1.0f);
        a.part_ml[(2ll * blockIdx.x + 1) * a.part_rows + lane] = make_float2(-INFINITY, -1.0f);
    }
    // warps that are ahead wait in the segments' ring for as long as one segment takes
    const long long seg_limit = span_limit((a.max_len + BN - 1) / BN);
    // the planner and its first segment, while the others set up
    if (warp == 4) {
        Walk walk(a, blockIdx.x == 0);
        bool more = walk.next();
        if (lane == 0) ring[0] = walk.s;
        ptx::tc_fence_before();
        __syncthreads();
        if (lane == 0) ptx::mbar_arrive(ctl.bar(L::bSegFull));
        bool ok = true;
        for (int q = 1; ok && more; ++q) {
            more = walk.next();
            const int k = q % kSegs;
            ok = ctl.warp_poll(L::bSegEmpty + k, ((q / kSegs) & 1) ^ 1, seg_limit);
            if (ok && lane == 0) {
                ring[k] = walk.s;
                ptx::mbar_arrive(ctl.bar(L::bSegFull + k));
            }
            __syncwarp();
        }
        __syncthreads();
        return;
    }
    if (warp == 2) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);

    // the rows around Q, while the first tiles are on their way (warps 0, 1, 3)
    auto clear_around_q = [&] {
        const int at = (warp == 3 ? 2 : warp) * 32 + lane;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        for (uint32_t e = at * 16; e < L::kQRows; e += 96 * 16) *reinterpret_cast<uint4*>(gbase + L::kZeros + e) = zero;
        for (int p = 0; p < 2 * L::kPanels; ++p)
            for (uint32_t e = L::kQRows + at * 16; e < L::kQPanel; e += 96 * 16)
                *reinterpret_cast<uint4*>(gbase + L::kQ0 + p * L::kQPanel + e) = zero;
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ctl.bar(L::bZeros));
    };

    // The q-th segment of this CTA, for one thread; false: a wait gave up.
    auto take = [&](int q, Seg& s) -> bool {
        if (!ctl.poll(L::bSegFull + q % kSegs, (q / kSegs) & 1, seg_limit)) return false;
        s = ring[q % kSegs];
        ptx::mbar_arrive(ctl.bar(L::bSegEmpty + q % kSegs));
        return true;
    };
    // The same for a whole warp: every field the same in every lane.
    auto warp_take = [&](int q, Seg& s) -> bool {
        if (!ctl.warp_poll(L::bSegFull + q % kSegs, (q / kSegs) & 1, seg_limit)) return false;
        const Seg r = ring[q % kSegs];
        s.row0 = uniform(r.row0);
        s.rows = uniform(r.rows);
        s.seq = uniform(r.seq);
        s.head = uniform(r.head);
        s.seen = uniform(r.seen);
        s.kt0 = uniform(r.kt0);
        s.n = uniform(r.n);
        s.part = uniform(r.part);
        if (lane == 0) ptx::mbar_arrive(ctl.bar(L::bSegEmpty + q % kSegs));
        return true;
    };

    if (warp >= 5) {
        // ------------------------------------------------------------ producers: Q and K, V
        const bool is_v = uniform(warp) == 6;
        if (elect_one()) {
            Feed<HD, true> feed{ctl, is_v ? &tmV : &tmK, is_v ? L::bFullV : L::bFullK,
                                is_v ? L::bEmptyV : L::bEmptyK, L::bLand, is_v,
                                base + (is_v ? L::kRingV : L::kRingK), RingPos(L::kSlots)};
            int q = 0;
            for (;; ++q) {
                Seg s;
                if (!take(q, s) || s.n == 0) break;
                if (!is_v) {
                    const int b = q & 1;
                    if (q >= 2 && !ctl.poll(L::bQEmpty + b, ((q >> 1) + 1) & 1)) break;
                    ptx::mbar_arrive_expect_tx(ctl.bar(L::bQFull + b),
                                               (uint32_t)(a.tile_rows * a.group * 128 * L::kPanels));
                    for (int p = 0; p < L::kPanels; ++p)
                        ptx::tma_load_3d(base + L::kQ0 + b * L::kQ + p * L::kQPanel, &tmQ, ctl.bar(L::bQFull + b), p * 64,
                                         s.head * a.group, s.row0);
                }
                if (!feed.tiles(a.table + (long long)s.seq * a.max_pages, a.page_shift, a.n_pages, s.kt0, s.n, s.seen,
                                s.head)) {
                    // Q lands before its K tiles are used, or here after a wait that gave up
                    if (!is_v) ptx::mbar_wait(ctl.bar(L::bQFull + (q & 1)), (q >> 1) & 1, kWaitLimit);
                    break;
                }
            }
            feed.drain();
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ MMA issuer
        if (elect_one()) {
            constexpr uint32_t idesc_qk = ptx::idesc_bf16(L::kM, BN, false, false);
            constexpr uint32_t idesc_pv = ptx::idesc_bf16(L::kM, HD, false, true);
            RingPos kp(L::kSlots), vp(L::kSlots);
            int steps[2] = {0, 0}, uses[2] = {0, 0};   // tiles and segments of each stream so far
            bool ok = ctl.poll(L::bZeros, 0);
            for (int q = 0; ok; ++q) {
                Seg s;
                if (!take(q, s) || s.n == 0) break;
                ok = ctl.poll(L::bQFull + (q & 1), (q >> 1) & 1);
                const uint32_t qd = desc_lo(base + L::kQ0 + (q & 1) * L::kQ, 16);
                // S0(0) S1(1) | PV(g) S(g+2) ... over the tiles g, stream g & 1
                for (int g = -2; ok && g < s.n; g += 2) {
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        const int v = g + st, k = g + st + 2;
                        if (v >= 0 && v < s.n) {
                            const int j = steps[st]++;
                            if (!ctl.poll(L::bFullV + vp.slot, vp.phase) || !ctl.poll(L::bPHalf + st, j & 1)) {
                                ok = false;
                                break;
                            }
                            // the segment's first P V overwrites O: its last one has been read
                            const bool fresh = v < 2;
                            if (fresh && uses[st] > 0 && !ctl.poll(L::bOEmpty + st, (uses[st] - 1) & 1)) {
                                ok = false;
                                break;
                            }
                            if (fresh) ++uses[st];
                            ptx::tc_fence_after();
                            const uint32_t vd = desc_lo(base + L::kRingV + vp.slot * L::kTile, kPanel);
                            const uint32_t to = tmem + tmem_o(st), tp = tmem + tmem_s(st) + kTmemP;
#pragma unroll
                            for (int kk = BN / 32; kk < BN / 16; ++kk)
                                mma_ts(to, tp + kk * 8, vd + kk * 128, idesc_pv, !fresh || kk > BN / 32);
                            if (!ctl.poll(L::bPFull + st, j & 1)) { ok = false; break; }
                            ptx::tc_fence_after();
#pragma unroll
                            for (int kk = 0; kk < BN / 32; ++kk)
                                mma_ts(to, tp + kk * 8, vd + kk * 128, idesc_pv, true);
                            ptx::mma_commit(ctl.bar(L::bEmptyV + vp.slot));
                            if (k >= s.n) ptx::mma_commit(ctl.bar(L::bOFull + st));
                            vp.advance();
                        }
                        if (k < s.n) {
                            if (!ctl.poll(L::bFullK + kp.slot, kp.phase)) { ok = false; break; }
                            ptx::tc_fence_after();
                            const uint32_t kd = desc_lo(base + L::kRingK + kp.slot * L::kTile, 16);
#pragma unroll
                            for (int kk = 0; kk < HD / 16; ++kk)
                                mma_ss(tmem + tmem_s(st), qd - st * (L::kQRows >> 4) + (((kk >> 2) * L::kQPanel + (kk & 3) * 32) >> 4),
                                       kd + (((kk >> 2) * kPanel + (kk & 3) * 32) >> 4), idesc_qk, kk > 0);
                            ptx::mma_commit(ctl.bar(L::bSFull + st));
                            ptx::mma_commit(ctl.bar(L::bEmptyK + kp.slot));
                            if (k == s.n - 1) ptx::mma_commit(ctl.bar(L::bQEmpty + (q & 1)));
                            kp.advance();
                        }
                    }
                }
            }
            // all MMAs of this CTA complete before TMEM is released
            ptx::mma_commit(ctl.bar(L::bFinal));
            ptx::mbar_wait(ctl.bar(L::bFinal), 0, kWaitLimit);
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------ V rows past the last key
        clear_around_q();
        int tiles = 0;
        uint32_t land_phase = 0;                       // by slot: parity of its next phase
        for (int q = 0;; ++q) {
            Seg s;
            if (!warp_take(q, s) || s.n == 0) break;
            tiles += s.n;
            const int live = s.seen - (s.kt0 + s.n - 1) * BN;
            if (live >= BN) continue;
            const int at = (tiles - 1) % L::kSlots;    // the segment's last V
            if (!ctl.warp_poll(L::bLand + at, (land_phase >> at) & 1u, seg_limit)) break;
            land_phase ^= 1u << at;
            uint8_t* v = gbase + L::kRingV + at * L::kTile;
            for (int e = live * 8 + lane; e < BN * 8; e += 32)
                for (int p = 0; p < L::kPanels; ++p)
                    *reinterpret_cast<uint4*>(v + p * kPanel + e * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async();               // ordered before the tensor core's reads
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ctl.bar(L::bFullV + at));
        }
    } else {
        // ------------------------------------------------------------ softmax of stream st
        const int st = uniform(warp);
        const uint32_t lane_off = (uint32_t)(st * 32) << 16;
        const uint32_t tS = tmem + lane_off + tmem_s(st), tO = tmem + lane_off + tmem_o(st);
        float* stage = reinterpret_cast<float*>(gbase) + lane * L::kStageRow;
        volatile float2* stage_ml = reinterpret_cast<volatile float2*>(gbase + L::kStageMl) + lane;
        clear_around_q();
        int done_steps = 0, uses = 0;
        for (int q = 0;; ++q) {
            Seg s;
            if (!warp_take(q, s) || s.n == 0) break;
            const int steps = (s.n + 1 - st) >> 1;
            const bool live = lane < s.rows * a.group;
            const int first = (s.kt0 + st) * BN;
            const int row = s.row0 + lane / a.group;
            // (0 for any limit below it: what follows subtracts key positions from it)
            int limit = s.seen;
            if (a.limits && live) limit = max(0, min(s.seen, __ldg(a.limits + row)));
            // steps whose tile every row sees whole; the rest is masked
            const int whole = __reduce_min_sync(0xFFFFFFFFu, limit) - first - BN;
            const int plain = whole < 0 ? 0 : min(steps, whole / (2 * BN) + 1);
            // lanes past the R rows hold no row: no logit passes their maximum
            float m = R == 32 || lane < R ? -INFINITY : INFINITY, l = 0.f;
            int j = 0;
            for (; j < steps; ++j) {
                if (!ctl.warp_poll(L::bSFull + st, (done_steps + j) & 1)) break;
                ptx::tc_fence_after();
                softmax_tile<HD, 0>(tS, j >= plain, limit - first - j * 2 * BN, a.scale_log2, m, l,
                                 ctl.bar(L::bPHalf + st));
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ctl.bar(L::bPFull + st));
            }
            if (j < steps) break;
            done_steps += steps;
            if (steps > 0) {
                if (!ctl.warp_poll(L::bOFull + st, uses & 1)) break;
                ++uses;
                ptx::tc_fence_after();
            }
            if (st == 1) {
                // ---- stream 1 hands its part over
                if (q > 0 && !ctl.warp_poll(L::bStageFree, (q - 1) & 1)) break;
                stage_ml->x = m;
                stage_ml->y = l;
                if (steps > 0) {
                    uint32_t o[HD];
                    load_row<HD>(tO, o);
                    if (live) {
#pragma unroll
                        for (int v = 0; v < HD / 4; ++v)
                            *reinterpret_cast<uint4*>(stage + 4 * v) =
                                make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                    }
                    ptx::tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) {
                    if (steps > 0) ptx::mbar_arrive(ctl.bar(L::bOEmpty + 1));
                    ptx::mbar_arrive(ctl.bar(L::bStage));
                }
                continue;
            }
            // ---- stream 0 adds the two: out = sum w O / sum w l, w = 2^(m - M)
            if (!ctl.warp_poll(L::bStage, q & 1)) break;
            const float m1 = stage_ml->x, l1 = stage_ml->y;
            const float M = fmaxf(m, m1);
            const float w0 = l != 0.f ? ptx::ex2(m - M) : 0.f, w1 = l1 != 0.f ? ptx::ex2(m1 - M) : 0.f;
            const float sum = w0 * l + w1 * l1;
            const bool whole_item = s.part < 0;
            const float scale = whole_item ? (sum != 0.f ? 1.0f / sum : 0.f) : 1.0f;
            const float f0 = w0 * scale, f1 = w1 * scale;
            __nv_bfloat16* orow = a.out + (long long)row * a.out_ld + (s.head * a.group + lane % a.group) * HD;
            const long long slot = 2ll * blockIdx.x + (whole_item ? 0 : s.part);
            float* prow = a.part_o + (slot * a.part_rows + lane) * HD;
            uint32_t o[HD];
            load_row<HD>(tO, o);
            if (live) {
                // a stream that saw no key has weight 0, and nothing in O or the stage
#pragma unroll
                for (int v = 0; v < HD / 4; ++v) {
                    const float4 y = f1 != 0.f ? *reinterpret_cast<const float4*>(stage + 4 * v) : make_float4(0.f, 0.f, 0.f, 0.f);
                    float x[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[e] = fmaf(f1, x[e], f0 != 0.f ? f0 * __uint_as_float(o[4 * v + e]) : 0.f);
                    if (whole_item)
                        *reinterpret_cast<uint2*>(orow + 4 * v) =
                            make_uint2(ptx::pack_bf16(x[0], x[1]), ptx::pack_bf16(x[2], x[3]));
                    else
                        *reinterpret_cast<float4*>(prow + 4 * v) = make_float4(x[0], x[1], x[2], x[3]);
                }
            }
            if (live && !whole_item) a.part_ml[slot * a.part_rows + lane] = make_float2(M, sum);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(ctl.bar(L::bOEmpty + 0));
                ptx::mbar_arrive(ctl.bar(L::bStageFree));
            }
        }
    }

    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 2) ptx::tmem_dealloc(tmem, 512);
}

// Adds the parts of the items that shares cut.  Block b looks at the boundary
// between CTA b and CTA b + 1; the blocks whose boundaries lie inside one item
// take its rows in turn.  One to eight warps per row, by the number of its
// parts: each adds some of them in the CTAs' order, then one adds the sums.
// (One block per item, a warp per row, took 50 us of 66 for 32 rows of 32 parts.)
template <int HD>
__global__ void __launch_bounds__(256)
paged_decode_merge_kernel(const __grid_constant__ Args a, int ctas) {
    constexpr int E = HD / 32;
    __shared__ float2 sum_ml[8];
    __shared__ float sum_o[8][HD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the lists are inputs: they may be read before the attention kernel is done
    SeqInfo mine = seq_info(a, lane, false);
    int total = __reduce_add_sync(0xFFFFFFFFu, mine.tiles);
    for (int k = 32; k < a.n_seqs; k += 32)
        total += __reduce_add_sync(0xFFFFFFFFu, seq_info(a, k + lane, false).tiles);
    const int c = (int)blockIdx.x + 1;
    // the item's rows and head, its parts, and where they lie: slot0, then 2 (base + p)
    int row0 = 0, rows = 0, head = 0, parts = 0, slot0 = 0, base = 0, turn = 0;
    const Shares sh(total * a.kv_heads, ctas);
    if (const int quota = item_quota(a, mine.tiles, sh, ctas)) {
        const ItemPart it(a, mine.tiles, quota, c);
        if (it.lane >= 0 && it.part > 0) {
            row0 = __shfl_sync(0xFFFFFFFFu, mine.row0, it.lane);
            rows = __shfl_sync(0xFFFFFFFFu, mine.rows, it.lane) * a.group;
            head = it.head;
            parts = it.parts;
            turn = it.part - 1;
            base = it.first;
            slot0 = 2 * base;
        }
    } else if (c < sh.n) {
        const int cut = sh.begin(c);
        for (int s0 = 0, at = 0; s0 < a.n_seqs; s0 += 32) {
            if (s0) mine = seq_info(a, s0 + lane, false);
            const int upto = warp_sum_to(mine.tiles);
            const int next = at + __shfl_sync(0xFFFFFFFFu, upto, 31) * a.kv_heads;
            if (cut < next) {
                const int from = at + (upto - mine.tiles) * a.kv_heads;
                const bool here = cut >= from && cut < from + mine.tiles * a.kv_heads;
                const int j = __ffs(__ballot_sync(0xFFFFFFFFu, here)) - 1;
                const int f = __shfl_sync(0xFFFFFFFFu, from, j);
                const int tiles = __shfl_sync(0xFFFFFFFFu, mine.tiles, j);
                head = (cut - f) / tiles;
                const int item = f + head * tiles;
                if (cut > item) {                              // inside the item, not its beginning
                    row0 = __shfl_sync(0xFFFFFFFFu, mine.row0, j);
                    rows = __shfl_sync(0xFFFFFFFFu, mine.rows, j) * a.group;
                    base = sh.owner(item);                     // its last part, then the first of the others
                    slot0 = 2 * base + 1;
                    parts = sh.owner(item + tiles - 1) - base + 1;
                    turn = c - base - 1;
                }
                break;
            }
            at = next;
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // the next call's kernel may set itself up; it waits for this one's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (rows == 0) return;
    auto slot_of = [&](int p) { return p == 0 ? (long long)slot0 : 2ll * (base + p); };
    const int width = parts <= 4 ? 1 : parts <= 8 ? 2 : parts <= 16 ? 4 : 8;      // warps per row
    const int per_block = 8 / width;
    // (every warp of the block makes the same number of rounds)
    for (int r0 = turn * per_block; r0 < rows; r0 += (parts - 1) * per_block) {
        const int r = r0 + warp / width;
        float M = -INFINITY, acc[E], sum = 0.f;
        bool missing = false;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
        auto add = [&](float2 ml, const float* src) {
            float x[E];
            if constexpr (E == 4) {
                const float4 v = *reinterpret_cast<const float4*>(src);
                x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
            } else {
                const float2 v = *reinterpret_cast<const float2*>(src);
                x[0] = v.x; x[1] = v.y;
            }
            missing = missing || ml.y < 0.f;
            if (ml.y != 0.f) {                                 // else the part saw no key
                const float top = fmaxf(M, ml.x);
                const float old = M > -INFINITY ? ptx::ex2(M - top) : 0.f, w = ptx::ex2(ml.x - top);
                sum = fmaf(w, ml.y, sum * old);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(w, x[e], acc[e] * old);
                M = top;
            }
        };
        if (r < rows) {
            // one pass, relative to the largest m so far: the loads of four parts are in flight together
#pragma unroll 4
            for (int p = warp % width; p < parts; p += width) {
                const long long at = slot_of(p) * a.part_rows + r;
                add(a.part_ml[at], a.part_o + at * HD + lane * E);
            }
        }
        if (width > 1) {
            if (lane == 0) sum_ml[warp] = make_float2(M, missing ? -1.f : sum);
#pragma unroll
            for (int e = 0; e < E; ++e) sum_o[warp][lane * E + e] = acc[e];
            __syncthreads();
            if (warp % width == 0)
                for (int p = 1; p < width; ++p) add(sum_ml[warp + p], &sum_o[warp + p][lane * E]);
            __syncthreads();
        }
        if (warp % width || r >= rows || missing) continue;    // missing: JANO_ETIMEOUT was raised
        const float inv = sum != 0.f ? 1.0f / sum : 0.f;
        __nv_bfloat16* dst = a.out + (long long)(row0 + r / a.group) * a.out_ld +
                             (head * a.group + r % a.group) * HD + lane * E;
        if constexpr (E == 4)
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(ptx::pack_bf16(acc[0] * inv, acc[1] * inv), ptx::pack_bf16(acc[2] * inv, acc[3] * inv));
        else
            *reinterpret_cast<uint32_t*>(dst) = ptx::pack_bf16(acc[0] * inv, acc[1] * inv);
    }
}

// Key tiles that the call's bounds allow.
long long max_tiles(const PagedAttentionCall& c) {
    const long long room = (long long)c.seqs->max_pages * c.pool->page_size;
    const long long len = c.max_len < room ? c.max_len : room;
    return ((len + BN - 1) / BN + 1) * c.seqs->n_seqs * c.pool->kv_heads;
}

template <int HD, int R>
cudaError_t launch_form(const PagedAttentionCall& c, Args& a, int ctas, cudaStream_t st) {
    using L = Layout<HD, R>;
    static DeviceOnce ready;
    int dev = 0;
    cudaGetDevice(&dev);
    if (!ready.done(dev)) {
        const cudaError_t e = cudaFuncSetAttribute(paged_decode_kernel<HD, R>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kAlloc);
        if (e != cudaSuccess) return e;
        ready.mark(dev);
    }
    a.tile_rows = R / a.group;
    CUtensorMap mq, mk, mv;
    if (!make_q_map(&mq, c.q, c.q_ld, c.n_rows, c.heads, HD, a.group, a.tile_rows) ||
        !make_pool_map(&mk, c.pool->k, *c.pool) || !make_pool_map(&mv, c.pool->v, *c.pool))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::kAlloc;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_decode_kernel<HD, R>, mq, mk, mv, a);
    if (e != cudaSuccess || ctas == 1) return e;
    cfg.gridDim = dim3((unsigned)(ctas - 1));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, paged_decode_merge_kernel<HD>, a, ctas);
}

}  // namespace

size_t paged_decode_workspace_bytes(int max_rows, int heads, int kv_heads, int d, int sms) {
    const long long rows = (long long)max_rows * (heads / kv_heads);
    if (rows > kMaxRows) return 0;
    return (size_t)2 * sms * rows * (d + 2) * sizeof(float);
}

bool paged_decode_fits(const PagedAttentionCall& c) { return max_tiles(c) <= 0x3FFFFFFF; }

cudaError_t launch_paged_decode(const PagedAttentionCall& c, int sms, int* err, cudaStream_t st) {
    Args a{};
    a.table = c.seqs->page_table;
    a.lens = c.seqs->seq_lens;
    a.cu = c.seqs->cu_rows;
    a.limits = c.limits;
    a.n_seqs = c.seqs->n_seqs;
    a.max_pages = c.seqs->max_pages;
    a.n_pages = c.pool->n_pages;
    while ((1 << a.page_shift) < c.pool->page_size) ++a.page_shift;
    a.n_rows = c.n_rows;
    a.max_rows = c.max_rows;
    const long long room = (long long)c.seqs->max_pages * c.pool->page_size;
    a.max_len = c.max_len < room ? c.max_len : (int)room;
    a.kv_heads = c.pool->kv_heads;
    a.group = c.heads / c.pool->kv_heads;
    a.scale_log2 = c.scale * 1.4426950408889634f;
    a.out = static_cast<__nv_bfloat16*>(c.out);
    a.out_ld = c.out_ld;
    a.part_rows = c.max_rows * a.group;
    a.part_ml = static_cast<float2*>(c.workspace);
    a.part_o = static_cast<float*>(c.workspace) + 4ll * sms * a.part_rows;
    a.err = err;
    // no more CTAs than key tiles that the bounds allow
    const long long most = max_tiles(c);
    const int ctas = (int)(most < sms ? most : sms);
    if (a.part_rows <= 16)
        return c.pool->d == 128 ? launch_form<128, 16>(c, a, ctas, st) : launch_form<64, 16>(c, a, ctas, st);
    return c.pool->d == 128 ? launch_form<128, 32>(c, a, ctas, st) : launch_form<64, 32>(c, a, ctas, st);
}

}  // namespace jano
