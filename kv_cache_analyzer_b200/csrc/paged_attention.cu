// paged_attention.cu -- attention of a chunk of rows of several sequences over
// their pages of a shared KV pool.
//
//   out[r, h] = sum_{j < L_r} softmax_j(scale * q[r,h] . k_j) v_j,
//   L_r = min(length of r's sequence, limits[r]),   0 where L_r <= 0,
//
// k_j, v_j at page page_table[s][j / page_size], place j % page_size, head
// h / G of the kv_heads (G = heads / kv_heads query heads share one).
//
// Flash-style on the 5th-generation tensor cores.  The G query heads of a row
// share K and V, so (row, head) pairs are packed into the 128 rows of an MMA
// tile: tile row p is query row p / G, head p % G of the group (128 / G whole
// query rows per tile).  A CTA runs two streams of (S = Q K^T, softmax,
// O += P V), one per softmax warpgroup, so the tensor core works on one while
// the other's exponentials run:
//   pair    two query tiles over the same key tiles (a sequence with more
//           rows than one tile holds): each K/V tile is read once for both;
//   single  one query tile, the even key tiles in stream 0 and the odd ones
//           in stream 1, each with its own running maximum, sum and O, merged
//           at the end: sequences of few rows, where the cache's bytes count
//           (64 rows each over 8 x 8,192 positions of 24 heads: 148 us, 5.4 TB/s).
// Which one a CTA takes is decided by its own sequence's rows, so one launch
// serves single tokens and long chunks together.
//
// Few rows leave SMs idle: the key tiles are then cut over the 2 to 8 CTAs
// of a thread-block cluster, which merge their (O, m, l) through distributed
// shared memory -- no workspace, no second launch, and a fixed order of sums.
// (At most 32 packed rows per sequence: paged_decode.cu, where a call brings
// a workspace.)
//
// Bound by the tensor core and the softmax together (58% of the cycles have an
// MMA) and by the rounds of CTAs over the SMs, and in long runs the card's power
// lowers the clock: 16,380 rows over 32,760 positions of 12 heads of 128, pages
// of 128 places, call after call, 3,101 us, 1,063 TFLOP/s (the contiguous kernel
// beside it 3,135 us, 1,052); after a pause 2,730 us.  Smaller pages
// are more copies: 4,096 rows over 16,384 positions of 24 heads take 753 us
// with pages of 256 places, 777 with 64, 818 with 16.
//
// 12 warps: 0-3 and 4-7 softmax warpgroups (thread = tile row = TMEM lane),
// 8 producer of Q and K, 9 MMA issuer, 10 clears V rows past the visible
// length (stale pages may hold NaN there, and 0 * NaN would reach O), 11
// producer of V.  A 128-key tile is gathered page by page: one box of
// min(page_size, 128) rows x 64 columns per page and panel.  The producers and
// the MMA issuer each run as one elected thread: elect.sync lets the compiler
// keep their operands in uniform registers, which halved the MMA thread's time
// per key tile.
// The pool's map has page, head and token strides of its own, so token-major
// and head-major pools, and K and V inside one allocation, read alike.
// TMEM columns: S0 [0,128) S1 [128,256) O0 [256,256+d) O1 [384,384+d); P_i is
// written over the upper half of S_i as BF16.
// Softmax statistics and O are fp32; P is rounded to BF16 (the type V has,
// which one MMA requires of both operands) and its sum l is taken before that
// rounding.  The running maximum follows lazily: O is rescaled only when it
// grows by more than 2^8, which keeps P within BF16's range either way.
// Every wait is bounded (the one that spans a CTA's key tiles by their number);
// a CTA that gives up records JANO_ETIMEOUT, takes part in the cluster's
// barriers, and the rows it shares are not written.
#include <cmath>

#include "paged_tile.cuh"

namespace jano {
namespace {

constexpr int kThreads = 384;
// As launched 384 x 168 registers; the softmax warpgroups hold a whole
// 128-column S row per thread.  2 x 128 x 208 + 128 x 80 <= 384 x 168.
constexpr int kRegsLaunch = 168;
constexpr int kRegsSoftmax = 208;
constexpr int kRegsIssue = 80;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsIssue <= kThreads * kRegsLaunch, "register split");
static_assert(2 * kRegsSoftmax + kRegsIssue <= 512, "sub-partition register file");
constexpr int kSoftmaxWarps = 8;
constexpr int kMaxSplit = 8;             // the portable cluster size; 16 ran twice as long as 8 in every shape

template <int HD>
struct Layout {
    static constexpr int kPanels = HD / 64;
    static constexpr int kSlots = HD == 64 ? 4 : 2;               // K tiles, and V tiles: 128 KB together
    static constexpr uint32_t kTile = kPanels * kPanel;           // Q, K or V tile bytes
    static constexpr uint32_t kQ1 = kTile;
    static constexpr uint32_t kRingK = 2 * kTile;
    static constexpr uint32_t kRingV = kRingK + kSlots * kTile;
    static constexpr uint32_t kBar = kRingV + kSlots * kTile;
    static constexpr int bQFull = 0;
    static constexpr int bFullK = 1;                   // [kSlots]
    static constexpr int bEmptyK = bFullK + kSlots;    // [kSlots]
    static constexpr int bFullV = bEmptyK + kSlots;    // [kSlots] landed and cleared past the last key
    static constexpr int bEmptyV = bFullV + kSlots;    // [kSlots]
    static constexpr int bLand = bEmptyV + kSlots;     // [kSlots] the ragged V tile landed, not yet cleared
    static constexpr int bSFull = bLand + kSlots;      // [2]
    static constexpr int bPFull = bSFull + 2;          // [2] whole P written
    static constexpr int bPHalf = bPFull + 2;          // [2] P of keys 64..127 written
    static constexpr int bOFull = bPHalf + 2;          // [2]
    static constexpr int bFinal = bOFull + 2;          // every MMA done
    static constexpr int kNumBars = bFinal + 1;
    static constexpr uint32_t kMisc = kBar + 8 * kNumBars;        // tmem base, abort, plan (12 ints)
    static constexpr uint32_t kMl = (kMisc + 64 + 15) / 16 * 16;  // float2 [2][128]: m, l of a tile row
    static constexpr uint32_t kBytes = kMl + 2 * BM * 8;
    static constexpr uint32_t kAlloc = kBytes + 1024;             // slack for 1 KB alignment
    static_assert(kAlloc <= 227 * 1024, "shared memory budget");
    // merge: fp32 O rows over Q and the ring, padded by 4 floats (16-byte
    // stores of adjacent rows fall on different banks)
    static constexpr uint32_t kRow = HD + 4;
    static constexpr uint32_t kWeights = 2 * BM * kRow * 4;        // then the rows' weights, float [256][2 * kMaxSplit]
    static_assert(kWeights + 2 * BM * 2 * kMaxSplit * 4 <= kBar, "merge buffer");
};

struct Args {
    const int32_t* table;
    const int32_t* lens;
    const int32_t* cu;
    const int32_t* limits;
    int n_seqs, max_pages, n_pages, page_shift;
    int n_rows, max_rows, max_len;
    int group, tile_rows;              // query heads per K/V head, query rows per tile
    int heads_first;                   // grid x is the K/V head, y the query tile pair
    float scale_log2;
    __nv_bfloat16* out;
    long long out_ld;
    int* err;
};

// What a CTA works on, from the device's lists; found by one warp.
struct Plan {
    int seq, row0, rows0, rows1, seen;   // rows of the two tiles, keys that any of them sees; rows0 = 0: nothing
};

// A sequence's rows and length, and its query tile pairs (0: none, or a bad one).
struct SeqRows {
    int lo, hi, len, tiles;
};
__device__ __forceinline__ SeqRows seq_rows(const Args& a, int s, bool report) {
    SeqRows q{0, 0, 0, 0};
    if (s >= a.n_seqs) return q;
    q.lo = __ldg(a.cu + s);
    q.hi = __ldg(a.cu + s + 1);
    q.len = __ldg(a.lens + s);
    const bool ok = q.lo >= 0 && q.lo <= q.hi && q.hi <= a.n_rows && q.hi - q.lo <= a.max_rows && q.len >= 0 &&
                    q.len <= a.max_len && (s > 0 || q.lo == 0);
    if (!ok && report) raise_error(a.err, JANO_EINDEX);
    const int step = 2 * a.tile_rows;
    if (ok) q.tiles = (q.hi - q.lo + step - 1) / step;
    return q;
}

// The x-th query tile pair of all sequences.  The longest of every 32
// sequences come first, so that the last CTAs to start are short ones, and the
// later tiles of a sequence before its earlier ones: under causal limits they
// see the most keys.
__device__ __forceinline__ Plan make_plan(const Args& a, int x, bool report) {
    const int lane = threadIdx.x & 31;
    Plan p{0, 0, 0, 0, 0};
    SeqRows q;
    int done = 0, s0 = 0;
    for (;; s0 += 32) {
        if (s0 >= a.n_seqs) return p;
        q = seq_rows(a, s0 + lane, report);
        const int all = __reduce_add_sync(0xFFFFFFFFu, q.tiles);
        if (x < done + all) break;
        done += all;
    }
    int before = 0;                            // tiles of the sequences that come first
    const int others = min(32, a.n_seqs - s0);
    for (int j = 0; j < others; ++j) {
        const int l = __shfl_sync(0xFFFFFFFFu, q.len, j), t = __shfl_sync(0xFFFFFFFFu, q.tiles, j);
        if (l > q.len || (l == q.len && j < lane)) before += t;
    }
    const unsigned who = __ballot_sync(0xFFFFFFFFu, x >= done + before && x < done + before + q.tiles);
    if (who) {
        const int src = __ffs(who) - 1;
        const int first = q.lo + (q.tiles - 1 - (x - (done + before))) * 2 * a.tile_rows;
        p.seq = s0 + src;
        p.row0 = __shfl_sync(0xFFFFFFFFu, first, src);
        const int left = __shfl_sync(0xFFFFFFFFu, q.hi - first, src);
        p.rows0 = min(left, a.tile_rows);
        p.rows1 = min(left - p.rows0, a.tile_rows);
        p.seen = __shfl_sync(0xFFFFFFFFu, q.len, src);
    }
    if (report)                                // the other sequences, for their errors
        for (int s = s0 + 32 + lane; s < a.n_seqs; s += 32) seq_rows(a, s, true);
    if (a.limits && p.rows0 > 0) {
        int most = 0;
        for (int i = lane; i < p.rows0 + p.rows1; i += 32) most = max(most, __ldg(a.limits + p.row0 + i));
        p.seen = min(p.seen, __reduce_max_sync(0xFFFFFFFFu, most));
    }
    return p;
}

// Parts of a tile row: one per CTA of the cluster, two (the streams) in the
// single form.  With M the largest m and w = 2^(m - M),
//   out = sum w O / sum w l,   summed in a fixed order.
// The rows are dealt over the cluster's CTAs.  First a thread per row reads the
// parts' (m, l) and leaves the weights w / sum in shared memory; then all
// softmax threads add 4 columns each (a warp per row, one after another, spent
// 1,500 cycles on each row's chain of remote reads).  The plan is read again
// from shared memory, so nothing of it is held through the loops.
template <int HD>
__device__ __forceinline__ void merge_rows(const Args& a) {
    using L = Layout<HD>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const volatile int* plan = reinterpret_cast<const volatile int*>(gbase + L::kMisc + 16);
    const int row0 = plan[1], rows0 = plan[2], rows1 = plan[3];
    const bool single = rows1 == 0;
    const int n_split = (int)gridDim.z, parts = single ? 2 * n_split : n_split;
    const int packed0 = rows0 * a.group, total = packed0 + rows1 * a.group;
    const int per = (total + n_split - 1) / n_split;
    const int begin = (int)blockIdx.z * per, count = min(per, total - begin);
    float* weight = reinterpret_cast<float*>(gbase + L::kWeights);     // [count][parts]
    const int t = threadIdx.x;
    // part c of packed row r: its (m, l) at slot(r, c), its O row there too
    auto slot = [&](int r, int c) {
        const int tile = r >= packed0;
        return (single ? c & 1 : tile) * BM + (tile ? r - packed0 : r);
    };
    auto peer = [&](int c) { return ptx::mapa_shared(base, (uint32_t)(single ? c >> 1 : c)); };
    if (t < count) {
        const int r = begin + t;
        float M = -INFINITY, sum = 0.f;
        bool missing = false;
        float* w = weight + t * parts;
        for (int c = 0; c < parts; ++c) {
            const float2 ml = ld_cluster_f2(peer(c) + L::kMl + slot(r, c) * 8);
            missing = missing || ml.y < 0.f;               // JANO_ETIMEOUT was raised
            // the sum so far is kept relative to the largest m so far
            const float top = fmaxf(M, ml.x);
            if (ml.y != 0.f) sum = (M > -INFINITY ? sum * ptx::ex2(M - top) : sum) + ml.y * ptx::ex2(ml.x - top);
            M = top;
            w[c] = ml.y != 0.f ? ml.x : -INFINITY;         // a part without visible keys has no O
        }
        const float inv = sum != 0.f ? 1.0f / sum : 0.f;
        for (int c = 0; c < parts; ++c)
            w[c] = missing ? -1.0f : (w[c] > -INFINITY || sum != sum ? ptx::ex2(w[c] - M) * inv : 0.f);
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");         // the softmax warps
    constexpr int kVec = HD / 4;
#pragma unroll 2
    for (int u = t; u < count * kVec; u += 32 * kSoftmaxWarps) {
        const int i = u / kVec, col = u % kVec, r = begin + i;
        const float* w = weight + i * parts;
        if (w[0] < 0.f) continue;
        float x0 = 0.f, x1 = 0.f, x2 = 0.f, x3 = 0.f;
#pragma unroll 4
        for (int c = 0; c < parts; ++c) {
            const float wc = w[c];
            if (wc != 0.f) {
                const float4 o = ld_cluster_f4(peer(c) + slot(r, c) * L::kRow * 4 + col * 16);
                x0 = fmaf(wc, o.x, x0);
                x1 = fmaf(wc, o.y, x1);
                x2 = fmaf(wc, o.z, x2);
                x3 = fmaf(wc, o.w, x3);
            }
        }
        const int tile = r >= packed0, p = tile ? r - packed0 : r;
        __nv_bfloat16* dst = a.out + (long long)(row0 + tile * a.tile_rows + p / a.group) * a.out_ld +
                             ((int)(a.heads_first ? blockIdx.x : blockIdx.y) * a.group + p % a.group) * HD + col * 4;
        *reinterpret_cast<uint2*>(dst) = make_uint2(ptx::pack_bf16(x0, x1), ptx::pack_bf16(x2, x3));
    }
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
paged_attention_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Args a) {
    using L = Layout<HD>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = a.heads_first ? blockIdx.x : blockIdx.y;      // K/V head
    const int n_split = (int)gridDim.z, split = (int)blockIdx.z;

    Ctl ctl;
    ctl.bar0 = base + L::kBar;
    ctl.abort = reinterpret_cast<volatile int*>(gbase + L::kMisc + 4);
    ctl.err = a.err;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::kMisc);
    int* plan_slot = reinterpret_cast<int*>(gbase + L::kMisc + 16);

    if (warp == 0) {
        const Plan p = make_plan(a, (int)(a.heads_first ? blockIdx.y : blockIdx.x),
                                 blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0);
        if (lane == 0) {
            plan_slot[0] = p.seq;
            plan_slot[1] = p.row0;
            plan_slot[2] = p.rows0;
            plan_slot[3] = p.rows1;
            plan_slot[4] = p.seen;
        }
    }
    if (threadIdx.x == 32) {
        ptx::mbar_init(ctl.bar(L::bQFull), 1);
        for (int s = 0; s < L::kSlots; ++s) {
            ptx::mbar_init(ctl.bar(L::bFullK + s), 1);
            ptx::mbar_init(ctl.bar(L::bEmptyK + s), 1);
            ptx::mbar_init(ctl.bar(L::bFullV + s), 1);
            ptx::mbar_init(ctl.bar(L::bEmptyV + s), 1);
            ptx::mbar_init(ctl.bar(L::bLand + s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(ctl.bar(L::bSFull + s), 1);
            ptx::mbar_init(ctl.bar(L::bPFull + s), 4);
            ptx::mbar_init(ctl.bar(L::bPHalf + s), 4);
            ptx::mbar_init(ctl.bar(L::bOFull + s), 1);
        }
        ptx::mbar_init(ctl.bar(L::bFinal), 1);
        *ctl.abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 8 && lane == 0) {
        ptx::prefetch_tmap(&tmQ);
        ptx::prefetch_tmap(&tmK);
        ptx::prefetch_tmap(&tmV);
    }
    if (warp == 9) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    // warp reductions tell the compiler that these are the same in every lane:
    // branches on them are uniform, and the MMAs take their descriptors and
    // addresses from uniform registers
    const uint32_t tmem = uniform(*tmem_slot);
    const int seq = uniform(plan_slot[0]), row0 = uniform(plan_slot[1]);
    const int rows0 = uniform(plan_slot[2]), rows1 = uniform(plan_slot[3]);
    const int seen = uniform(max(plan_slot[4], 0));
    const bool single = rows1 == 0;
    // this CTA's key tiles [kt0, kt0 + n); n steps per stream in the pair
    // form, ceil(n / 2) and floor(n / 2) in the single form
    const int nt = (seen + BN - 1) / BN;
    const int kt0 = (int)((long long)nt * split / n_split);
    const int n = rows0 > 0 ? (int)((long long)nt * (split + 1) / n_split) - kt0 : 0;
    const bool ragged = n > 0 && kt0 + n == nt && seen % BN != 0;   // this CTA holds the ragged last tile
    const bool merge = rows0 > 0 && (single || n_split > 1);

    if (warp >= 8) {
      ptx::setmaxnreg_dec<kRegsIssue>();
      if ((warp == 8 || warp == 11) && n > 0) {
        // ------------------------------------------------------------ producers: Q and K, V
        const bool is_v = uniform(warp) == 11;
        if (elect_one()) {
            if (!is_v) {
                const uint32_t q_bytes = (uint32_t)(a.tile_rows * a.group * 128 * L::kPanels);
                ptx::mbar_arrive_expect_tx(ctl.bar(L::bQFull), single ? q_bytes : 2 * q_bytes);
                for (int p = 0; p < L::kPanels; ++p) {
                    ptx::tma_load_3d(base + p * kPanel, &tmQ, ctl.bar(L::bQFull), p * 64, head * a.group, row0);
                    if (!single)
                        ptx::tma_load_3d(base + L::kQ1 + p * kPanel, &tmQ, ctl.bar(L::bQFull), p * 64, head * a.group,
                                         row0 + a.tile_rows);
                }
            }
            Feed<HD, false> feed{ctl, is_v ? &tmV : &tmK, is_v ? L::bFullV : L::bFullK,
                                 is_v ? L::bEmptyV : L::bEmptyK, L::bLand, is_v,
                                 base + (is_v ? L::kRingV : L::kRingK), RingPos(L::kSlots)};
            feed.tiles(a.table + (long long)seq * a.max_pages, a.page_shift, a.n_pages, kt0, n, seen, head);
            if (!is_v) ptx::mbar_wait(ctl.bar(L::bQFull), 0, kWaitLimit);
            feed.drain();
        }
      } else if (warp == 9 && n > 0) {
        // ------------------------------------------------------------ MMA issuer
        if (elect_one()) {
            constexpr uint32_t idesc_qk = ptx::idesc_bf16(BM, BN, false, false);
            constexpr uint32_t idesc_pv = ptx::idesc_bf16(BM, HD, false, true);
            RingPos kp(L::kSlots), vp(L::kSlots);
            auto wait_k = [&]() { return ctl.poll(L::bFullK + kp.slot, kp.phase); };
            auto wait_v = [&]() { return ctl.poll(L::bFullV + vp.slot, vp.phase); };
            auto release_k = [&]() { ptx::mma_commit(ctl.bar(L::bEmptyK + kp.slot)); kp.advance(); };
            auto release_v = [&]() { ptx::mma_commit(ctl.bar(L::bEmptyV + vp.slot)); vp.advance(); };
            auto qk = [&](int st, uint32_t qb) {           // S_st = Q K^T, K the ring's next tile
                const uint32_t kd = desc_lo(base + L::kRingK + kp.slot * L::kTile, 16), qd = desc_lo(qb, 16);
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * kPanel + (kk & 3) * 32) >> 4;
                    mma_ss(tmem + tmem_s(st), qd + off, kd + off, idesc_qk, kk > 0);
                }
                ptx::mma_commit(ctl.bar(L::bSFull + st));
            };
            // O_st += P_st V over key sixteenths [k0, k1); V the ring's next tile
            auto pv = [&](int st, int k0, int k1, bool acc) {
                const uint32_t vd = desc_lo(base + L::kRingV + vp.slot * L::kTile, kPanel);
#pragma unroll
                for (int kk = k0; kk < k1; ++kk)
                    mma_ts(tmem + tmem_o(st), tmem + tmem_s(st) + kTmemP + kk * 8, vd + kk * 128, idesc_pv,
                           acc || kk > k0);
            };
            auto pv_tile = [&](int st, int j) -> bool {    // its j-th tile
                if (!ctl.poll(L::bPHalf + st, j & 1)) return false;
                ptx::tc_fence_after();
                pv(st, BN / 32, BN / 16, j > 0);
                if (!ctl.poll(L::bPFull + st, j & 1)) return false;
                ptx::tc_fence_after();
                pv(st, 0, BN / 32, true);
                return true;
            };
            bool ok = ctl.poll(L::bQFull, 0);
            if (!single) {
                // S0_0 S1_0 | PV0_{j-1} S0_j PV1_{j-1} S1_j | ... PV0 PV1
                if (ok && (ok = wait_k())) {
                    ptx::tc_fence_after();
                    qk(0, base);
                    qk(1, base + L::kQ1);
                    release_k();
                }
                for (int j = 1; ok && j < n; ++j) {
                    if (!wait_v() || !wait_k()) { ok = false; break; }
                    if (!pv_tile(0, j - 1)) { ok = false; break; }
                    qk(0, base);
                    if (!pv_tile(1, j - 1)) { ok = false; break; }
                    release_v();
                    qk(1, base + L::kQ1);
                    release_k();
                }
                if (ok) {
                    ok = wait_v() && pv_tile(0, n - 1);
                    if (ok) {
                        ptx::mma_commit(ctl.bar(L::bOFull + 0));
                        ok = pv_tile(1, n - 1);
                    }
                    if (ok) {
                        ptx::mma_commit(ctl.bar(L::bOFull + 1));
                        release_v();
                    }
                }
            } else {
                // S0(0) S1(1) | PV(g) S(g+2) ... over the tiles g, stream g & 1
                for (int g = -2; ok && g < n; g += 2) {
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        const int v = g + st, k = g + st + 2;
                        if (v >= 0 && v < n) {
                            if (!wait_v() || !pv_tile(st, v >> 1)) { ok = false; break; }
                            release_v();
                            if (k >= n) ptx::mma_commit(ctl.bar(L::bOFull + st));
                        }
                        if (k < n) {
                            if (!wait_k()) { ok = false; break; }
                            ptx::tc_fence_after();
                            qk(st, base);
                            release_k();
                        }
                    }
                }
            }
            // all MMAs of this CTA complete before TMEM or shared memory is reused
            ptx::mma_commit(ctl.bar(L::bFinal));
            ptx::mbar_wait(ctl.bar(L::bFinal), 0, kWaitLimit);
        }
      } else if (warp == 10 && ragged) {
        // ------------------------------------------------------------ V rows past the last key
        const int at = (n - 1) % L::kSlots;
        if (ctl.warp_wait(L::bLand + at, 0, span_limit(n))) {
            const int live = seen - (nt - 1) * BN;
            uint8_t* v = gbase + L::kRingV + at * L::kTile;
            for (int e = live * 8 + lane; e < BN * 8; e += 32)
                for (int p = 0; p < L::kPanels; ++p)
                    *reinterpret_cast<uint4*>(v + p * kPanel + e * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async();           // ordered before the tensor core's reads
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ctl.bar(L::bFullV + at));
        }
      }
      // the same barriers as the softmax warps' (both branches end for
      // themselves: where they met again, the register counts would differ)
      __syncwarp();
      if (merge) {
        if (n_split > 1) {
            ptx::cluster_sync_all();
            ptx::cluster_sync_all();
        } else {
            __syncthreads();
        }
      }
      __syncthreads();
      ptx::tc_fence_after();
      if (warp == 9) ptx::tmem_dealloc(tmem, 512);
    } else {
        ptx::setmaxnreg_inc<kRegsSoftmax>();
        // ------------------------------------------------------------ softmax WG i
        const int i = uniform(warp >> 2);
        const int q = uniform(warp & 3);              // TMEM lane quarter of this warp
        const int row = q * 32 + lane;
        const uint32_t lane_off = (uint32_t)(q * 32) << 16;
        const uint32_t tS = tmem + lane_off + tmem_s(i);
        const uint32_t tO = tmem + lane_off + tmem_o(i);
        const bool warp_live = q * 32 < (i && !single ? rows1 : rows0) * a.group;   // else only the barriers are kept
        const int steps = single ? (n + 1 - i) >> 1 : n;
        // the stream's tiles start at keys first, first + apart, ...
        const int first = (kt0 + (single ? i : 0)) * BN, apart = single ? 2 * BN : BN;
        // (0 for any limit below it: what follows subtracts key positions from it)
        int limit = seen;
        if (a.limits && row < (i && !single ? rows1 : rows0) * a.group)
            limit = max(0, min(seen, __ldg(a.limits + row0 + (i && !single ? a.tile_rows : 0) + row / a.group)));
        // steps whose tile every row of the warp sees whole; the rest is masked
        const int whole = __reduce_min_sync(0xFFFFFFFFu, limit) - first - BN;
        const int plain = whole < 0 ? 0 : min(steps, whole / apart + 1);
        float m = -INFINITY, l = 0.f;
        int j = 0;
        if (warp_live) {
            constexpr int kPolyEighths = HD == 64 ? 3 : 0;
            // (two loops: the one body with a branch in it cost 4% of a long chunk's time)
            for (; j < plain; ++j) {
                if (!ctl.warp_wait(L::bSFull + i, j & 1)) break;
                ptx::tc_fence_after();
                softmax_tile<HD, kPolyEighths>(tS, false, BN, a.scale_log2, m, l, ctl.bar(L::bPHalf + i));
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ctl.bar(L::bPFull + i));
            }
            for (; j < steps; ++j) {
                if (!ctl.warp_wait(L::bSFull + i, j & 1)) break;
                ptx::tc_fence_after();
                softmax_tile<HD, 0>(tS, true, limit - first - j * apart, a.scale_log2, m, l, ctl.bar(L::bPHalf + i));
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ctl.bar(L::bPFull + i));
            }
        } else {
            for (; j < steps; ++j) {
                if (!ctl.warp_wait(L::bSFull + i, j & 1)) break;
                if (lane == 0) {
                    ptx::mbar_arrive(ctl.bar(L::bPHalf + i));
                    ptx::mbar_arrive(ctl.bar(L::bPFull + i));
                }
            }
        }
        const bool ok = j == steps;
        const int tile = i && !single ? 1 : 0;
        const int qrow = row0 + tile * a.tile_rows + row / a.group;
        const bool live = row < (tile ? rows1 : rows0) * a.group;
        // ------------------------------------------------------------ epilogue
        // before a merge every MMA of the CTA is done: O goes where they read
        bool done = ok;
        if (done && n > 0) done = ctl.warp_wait(merge ? L::bFinal : L::bOFull + i, 0) && !*ctl.abort;
        ptx::tc_fence_after();
        if (merge) {
            float2* ml = reinterpret_cast<float2*>(gbase + L::kMl) + i * BM + row;
            // l < 0 (impossible for a sum of exponentials) marks a part that is missing
            *ml = done ? make_float2(m, l) : make_float2(-INFINITY, -1.0f);
            if (done && steps > 0 && warp_live) {
                float* po = reinterpret_cast<float*>(gbase) + (i * BM + row) * L::kRow;
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    uint32_t o[32];
                    ptx::tmem_ld32(tO + 32 * c, o);
                    ptx::tmem_wait_ld();
                    if (live) {
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            *reinterpret_cast<float4*>(po + 32 * c + 4 * v) =
                                make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                            __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
                    }
                }
            }
        } else if (done && warp_live) {
            const float inv = l != 0.f ? 1.0f / l : 0.f;      // a row that saw no key: 0
            __nv_bfloat16* orow = a.out + (long long)qrow * a.out_ld + (head * a.group + row % a.group) * HD;
#pragma unroll
            for (int c = 0; c < HD / 32; ++c) {
                uint32_t o[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0u;
                if (steps > 0) {
                    ptx::tmem_ld32(tO + 32 * c, o);
                    ptx::tmem_wait_ld();
                }
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    pk[e] = ptx::pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                if (live) {
                    uint4* dst = reinterpret_cast<uint4*>(orow + 32 * c);
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        dst[v] = make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
                }
            }
        }
        // ------------------------------------------------------------ merge
        if (merge) {
            __syncwarp();
            if (n_split > 1) ptx::cluster_sync_all();
            else __syncthreads();
            merge_rows<HD>(a);
            // no CTA leaves while a peer may still read its shared memory
            __syncwarp();
            if (n_split > 1) ptx::cluster_sync_all();
        }
        ptx::tc_fence_before();
        __syncthreads();
    }
}

template <int HD>
cudaError_t set_up(int dev) {
    using L = Layout<HD>;
    static DeviceOnce ready;
    if (ready.done(dev)) return cudaSuccess;
    // the register split assumes exactly kRegsLaunch registers per thread
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, paged_attention_kernel<HD>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(paged_attention_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kAlloc);
    if (e == cudaSuccess) ready.mark(dev);
    return e;
}

template <int HD>
cudaError_t launch_hd(const PagedAttentionCall& c, const Args& a, int tiles, int* err, cudaStream_t st) {
    using L = Layout<HD>;
    int dev = 0;
    cudaGetDevice(&dev);
    const cudaError_t e = set_up<HD>(dev);
    if (e != cudaSuccess) return e;
    int sms = 148;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    int split = c.n_split;
    if (split == 0)
        split = paged_split_count(c.n_rows, c.max_rows, c.max_len, c.seqs->n_seqs, c.heads, c.pool->kv_heads, sms);
    CUtensorMap mq, mk, mv;
    if (!make_q_map(&mq, c.q, c.q_ld, c.n_rows, c.heads, HD, a.group, a.tile_rows) ||
        !make_pool_map(&mk, c.pool->k, *c.pool) || !make_pool_map(&mv, c.pool->v, *c.pool))
        return cudaErrorInvalidValue;
    const dim3 grid = a.heads_first ? dim3((unsigned)c.pool->kv_heads, (unsigned)tiles, (unsigned)split)
                                    : dim3((unsigned)tiles, (unsigned)c.pool->kv_heads, (unsigned)split);
    if (split == 1) {
        paged_attention_kernel<HD><<<grid, kThreads, L::kAlloc, st>>>(mq, mk, mv, a);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::kAlloc;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {1, 1, (unsigned)split};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_attention_kernel<HD>, mq, mk, mv, a);
}

// Query tile pairs that n_seqs sequences of at most max_rows rows, n_rows in
// all, can have at most.
long long tile_bound(int n_rows, int max_rows, int n_seqs, int tile_rows) {
    const long long step = 2ll * tile_rows;
    const long long each = (max_rows + step - 1) / step * (long long)n_seqs;
    const long long all = n_rows / step + n_seqs;
    return each < all ? each : all;
}

}  // namespace

// CTAs per (query tile pair, K/V head): the cluster size z (1, 2, 4, 8) with
// the shortest modelled time: rounds of the C clusters over the device times
// the key tiles of one CTA plus the equivalent of 5 tiles for its set-up, fill
// and drain, 7.5 where a merge follows (1.8 us a tile).  Clusters of 4 and 8 do
// not fill the GPCs: 33 of 37 and 15 of 18 are resident at once on 148 SMs.
// Over 17 measured shapes (1 to 768 CTAs, 3 to 591 key tiles) the choice is
// within 6% of the best.
int paged_split_count(int n_rows, int max_rows, int max_len, int n_seqs, int heads, int kv_heads, int sms) {
    if (n_rows <= 0 || max_rows <= 0 || max_len <= 0 || sms <= 0) return 1;
    const int tile_rows = BM / (heads / kv_heads);
    const long long clusters = tile_bound(n_rows, max_rows, n_seqs, tile_rows) * kv_heads;
    const int nt = (max_len + BN - 1) / BN;
    int best = 1;
    double best_t = 0.0;
    for (int z = 1; z <= kMaxSplit && z <= nt; z *= 2) {
        const int fit = sms / z - (z == 4 ? sms / 37 : z == 8 ? sms / 49 : 0);
        const long long resident = fit < 1 ? 1 : fit;
        const double rounds = (double)((clusters + resident - 1) / resident);
        const double t = rounds * ((double)nt / z + (z == 1 ? 5.0 : 7.5));
        if (z == 1 || t < best_t * (1.0 - 1e-9)) {
            best_t = t;
            best = z;
        }
    }
    return best;
}

cudaError_t launch_paged_attention(const PagedAttentionCall& c, int* err, cudaStream_t st) {
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
    // a longer sequence than the table can describe is reported like one above max_len
    const long long room = (long long)c.seqs->max_pages * c.pool->page_size;
    a.max_len = c.max_len < room ? c.max_len : (int)room;
    a.group = c.heads / c.pool->kv_heads;
    a.tile_rows = BM / a.group;
    a.scale_log2 = c.scale * 1.4426950408889634f;
    a.out = static_cast<__nv_bfloat16*>(c.out);
    a.out_ld = c.out_ld;
    a.err = err;
    const long long tiles = tile_bound(c.n_rows, c.max_rows, c.seqs->n_seqs, a.tile_rows);
    if (tiles > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    // One sequence: its tiles side by side, so that the CTAs at work share the
    // K/V of few heads in L2 (4,680 rows over 32,760 positions: 915 us, heads
    // first 1,048).  Several: all heads of the longest tiles first, so that the
    // last CTAs are short ones (eight sequences of 500 to 8,000 positions: 440
    // us, tiles first 485; the due sets of three images, after a pause: 144 and
    // 151).
    a.heads_first = c.seqs->n_seqs > 1 && tiles <= 65535;
    return c.pool->d == 128 ? launch_hd<128>(c, a, (int)tiles, err, st) : launch_hd<64>(c, a, (int)tiles, err, st);
}

}  // namespace jano
