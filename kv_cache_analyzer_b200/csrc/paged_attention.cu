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
//           at the end.  This is the form of single tokens, bound by the
//           cache's bytes: up to four K/V tiles (128 KB for d = 128) are in
//           flight per SM, and half-empty MMA tiles cost nothing that counts.
// Which one a CTA takes is decided by its own sequence's rows, so one launch
// serves single tokens and long chunks together.
//
// Few rows leave SMs idle: the key tiles are then cut over the 2 to 16 CTAs
// of a thread-block cluster, which merge their (O, m, l) through distributed
// shared memory -- no workspace, no second launch, and a fixed order of sums.
//
// 12 warps: 0-3 and 4-7 softmax warpgroups (thread = tile row = TMEM lane),
// 8 TMA producer, 9 MMA issuer, 10 clears V rows past the visible length
// (stale pages may hold NaN there, and 0 * NaN would reach O), 11 idle.  A
// 128-key tile is gathered page by page: one box of min(page_size, 128) rows
// x 64 columns per page and panel.  The producer and the MMA issuer each run as
// one elected thread: elect.sync lets the compiler keep their operands in
// uniform registers, which halved the MMA thread's time per key tile.
// The pool's map has page, head and token strides of its own, so token-major
// and head-major pools, and K and V inside one allocation, read alike.
// TMEM columns: S0 [0,128) S1 [128,256) O0 [256,256+d) O1 [384,384+d); P_i is
// written over the upper half of S_i as BF16.
// Softmax statistics and O are fp32; P is rounded to BF16 (the type V has,
// which one MMA requires of both operands) and its sum l is taken before that
// rounding.  The running maximum follows lazily: O is rescaled only when it
// grows by more than 2^8, which keeps P within BF16's range either way.
// Every wait is bounded; a CTA that gives up records JANO_ETIMEOUT, takes
// part in the cluster's barriers, and the rows it shares are not written.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <mutex>

#include "jano_common.cuh"

namespace jano {
namespace {

constexpr int BM = 128;            // tile rows
constexpr int BN = 128;            // keys per tile
constexpr int kThreads = 384;
// As launched 384 x 168 registers; the softmax warpgroups hold a whole
// 128-column S row per thread.  2 x 128 x 208 + 128 x 80 <= 384 x 168.
constexpr int kRegsLaunch = 168;
constexpr int kRegsSoftmax = 208;
constexpr int kRegsIssue = 80;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsIssue <= kThreads * kRegsLaunch, "register split");
static_assert(2 * kRegsSoftmax + kRegsIssue <= 512, "sub-partition register file");
constexpr uint32_t kPanel = 128 * 128;       // bytes of one 128-row x 64-column panel
constexpr int kSoftmaxWarps = 8;
constexpr int kMaxSplit = 16;
constexpr int kMaxBoxes = 8;         // pages of 16 rows in a 128-key tile
constexpr long long kWaitLimit = 1ll << 31;  // cycles (~1 s)

template <int HD>
struct Layout {
    static constexpr int kPanels = HD / 64;
    static constexpr int kSlots = HD == 64 ? 8 : 4;               // 128 KB of K/V tiles
    static constexpr uint32_t kTile = kPanels * kPanel;           // Q, K or V tile bytes
    static constexpr uint32_t kQ1 = kTile;
    static constexpr uint32_t kRing = 2 * kTile;
    static constexpr uint32_t kBar = kRing + kSlots * kTile;
    static constexpr int bQFull = 0;
    static constexpr int bFull = 1;                    // [kSlots] tile in shared memory, V cleared
    static constexpr int bEmpty = bFull + kSlots;      // [kSlots]
    static constexpr int bSFull = bEmpty + kSlots;     // [2]
    static constexpr int bPFull = bSFull + 2;          // [2] whole P written
    static constexpr int bPHalf = bPFull + 2;          // [2] P of keys 64..127 written
    static constexpr int bOFull = bPHalf + 2;          // [2]
    static constexpr int bLast = bOFull + 2;           // the ragged V tile landed, not yet cleared
    static constexpr int bFinal = bLast + 1;           // every MMA done
    static constexpr int kNumBars = bFinal + 1;
    static constexpr uint32_t kMisc = kBar + 8 * kNumBars;        // tmem base, abort, plan (12 ints)
    static constexpr uint32_t kMl = (kMisc + 64 + 15) / 16 * 16;  // float2 [2][128]: m, l of a tile row
    static constexpr uint32_t kBytes = kMl + 2 * BM * 8;
    static constexpr uint32_t kAlloc = kBytes + 1024;             // slack for 1 KB alignment
    static_assert(kAlloc <= 227 * 1024, "shared memory budget");
    // merge: fp32 O rows over Q and the ring, padded by 4 floats (16-byte
    // stores of adjacent rows fall on different banks)
    static constexpr uint32_t kRow = HD + 4;
    static_assert(2 * BM * kRow * 4 <= kBar, "merge buffer");
    __host__ __device__ static constexpr uint32_t tS(int i) { return i ? 128u : 0u; }
    __host__ __device__ static constexpr uint32_t tO(int i) { return i ? 384u : 256u; }
    static constexpr uint32_t tP = 64;                             // offset of P inside S
};

struct Args {
    const int32_t* table;
    const int32_t* lens;
    const int32_t* cu;
    const int32_t* limits;
    int n_seqs, max_pages, n_pages, page_shift;
    int n_rows, max_rows, max_len;
    int group, tile_rows;              // query heads per K/V head, query rows per tile
    float scale_log2;
    __nv_bfloat16* out;
    long long out_ld;
    int* err;
};

struct Ctl {
    uint32_t bar0;
    volatile int* abort;
    int* err;
    __device__ uint32_t bar(int i) const { return bar0 + 8u * (uint32_t)i; }
    // Waiting threads sleep until the phase completes; the MMA warp polls
    // (its waits sit on every key tile's critical path).
    __device__ bool wait(int i, uint32_t parity) const {
        if (ptx::mbar_try_wait_sleep(bar(i), parity)) return true;
        const long long t0 = clock64();
        for (;;) {
            if (ptx::mbar_try_wait_sleep(bar(i), parity)) return true;
            if (*abort) return false;
            if (clock64() - t0 > kWaitLimit) {
                *abort = 1;
                raise_error(err, JANO_ETIMEOUT);
                return false;
            }
        }
    }
    __device__ bool poll(int i, uint32_t parity) const {
        if (ptx::mbar_try_wait(bar(i), parity)) return true;
        const long long t0 = clock64();
        while (!ptx::mbar_try_wait(bar(i), parity)) {
            if (*abort) return false;
            if (clock64() - t0 > kWaitLimit) {
                *abort = 1;
                raise_error(err, JANO_ETIMEOUT);
                return false;
            }
        }
        return true;
    }
    // Warp-uniform: the .sync.aligned operations that follow never diverge.
    __device__ bool warp_wait(int i, uint32_t parity) const {
        int ok = 0;
        if ((threadIdx.x & 31) == 0) ok = wait(i, parity) ? 1 : 0;
        return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
    }
};

__device__ __forceinline__ int uniform(int v) { return __reduce_max_sync(0xFFFFFFFFu, v); }
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_max_sync(0xFFFFFFFFu, v); }
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3) : "memory");
}
// Shared-memory operand descriptors as two words, so that stepping through a
// tile is one 32-bit add: the low word holds address / 16 and the leading
// offset, the high word (stride 1024, 128-byte swizzle) is the same for all.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// (the mask drops the CTA rank that a shared address carries inside a cluster)
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) {
    return ((addr >> 4) & 0x3FFFu) | ((lead >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool acc) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\t"
                 "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}"
                 ::"r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"((uint32_t)acc) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool acc) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}"
                 ::"r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"((uint32_t)acc) : "memory");
}
// One lane of the converged warp, chosen by the hardware: unlike lane == 0 it
// tells the compiler that a single thread runs what follows.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// Order of the K and V loads of a CTA with n key tiles, and the load index of
// tile g's K and V.
//   pair:   K0 V0 K1 V1 ...         single: K0 K1 V0 K2 V1 K3 ... V(n-1)
// (in the single form two tiles' S are in work at once, one per stream).
struct LoadOrder {
    bool single;
    int n;
    __device__ int k(int g) const { return single ? (g < 2 ? g : 2 * g - 1) : 2 * g; }
    __device__ int v(int g) const { return single ? min(2 * g + 2, 2 * n - 1) : 2 * g + 1; }
    // tile of load i, and whether it is a V
    __device__ int tile(int i, bool& is_v) const {
        if (!single) {
            is_v = i & 1;
            return i >> 1;
        }
        if (i < 2) {
            is_v = n == 1 && i == 1;
            return is_v ? 0 : i;
        }
        is_v = i == 2 * n - 1 || !(i & 1);
        return i == 2 * n - 1 ? n - 1 : (is_v ? (i - 2) >> 1 : (i + 1) >> 1);
    }
};

// Row max of 64 values; with kMask, keys >= valid are left out.
template <bool kMask>
__device__ __forceinline__ float max64(const uint32_t (&s)[64], int valid) {
    float m[8];
#pragma unroll
    for (int a = 0; a < 8; ++a) m[a] = -INFINITY;
#pragma unroll
    for (int e = 0; e < 64; e += 2) {
        float x = __uint_as_float(s[e]), y = __uint_as_float(s[e + 1]);
        if (kMask && e >= valid) x = -INFINITY;
        if (kMask && e + 1 >= valid) y = -INFINITY;
        m[(e >> 1) & 7] = ptx::fmax3(m[(e >> 1) & 7], x, y);
    }
    return fmaxf(ptx::fmax3(m[0], m[1], m[2]), ptx::fmax3(m[3], m[4], fmaxf(m[5], fmaxf(m[6], m[7]))));
}

// p = 2^(s*c - m) for 64 values, packed to 32 BF16x2 words; returns sum(p).
// Masked keys give exactly 0, whatever S holds there.
template <bool kMask>
__device__ __forceinline__ float exp64(const uint32_t (&s)[64], int valid, float c, float m, uint32_t* pk) {
    const uint64_t c2 = ptx::f2(c, c), nm2 = ptx::f2(-m, -m);
    uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
    for (int e = 0; e < 64; e += 2) {
        float xa, xb;
        ptx::f2split(ptx::ffma2(ptx::f2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, nm2), xa, xb);
        float a = ptx::ex2(xa), b = ptx::ex2(xb);
        if (kMask && e >= valid) a = 0.f;
        if (kMask && e + 1 >= valid) b = 0.f;
        acc[(e >> 1) & 3] = ptx::fadd2(acc[(e >> 1) & 3], ptx::f2(a, b));
        pk[e >> 1] = ptx::pack_bf16(a, b);
    }
    float lo, hi;
    ptx::f2split(ptx::fadd2(ptx::fadd2(acc[0], acc[1]), ptx::fadd2(acc[2], acc[3])), lo, hi);
    return lo + hi;
}

// One key tile of one tile row (see the file comment): S from TMEM, maximum,
// lazy rescale of O, P back as BF16.  `valid`: keys of the tile this row sees.
template <int HD, bool kMask>
__device__ __forceinline__ void softmax_tile(uint32_t tS, int valid, float c, float& m, float& l, uint32_t bar_half) {
    constexpr uint32_t kO = Layout<HD>::tO(0) - Layout<HD>::tS(0);      // the same for both streams
    static_assert(Layout<HD>::tO(1) - Layout<HD>::tS(1) == kO, "O lies at one distance from S");
    const uint32_t tO = tS + kO, tP = tS + Layout<HD>::tP;
    uint32_t s[128];
    ptx::tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
    ptx::tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
    ptx::tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&s[64]));
    ptx::tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&s[96]));
    ptx::tmem_wait_ld();
    const uint32_t(&lo)[64] = *reinterpret_cast<const uint32_t(*)[64]>(&s[0]);
    const uint32_t(&hi)[64] = *reinterpret_cast<const uint32_t(*)[64]>(&s[64]);
    const float mxs = fmaxf(max64<kMask>(lo, valid), max64<kMask>(hi, valid - 64)) * c;
    // a row that has seen no key yet keeps m = -inf: its P is masked to 0
    const bool want = mxs > m + 8.0f;
    if (__any_sync(0xFFFFFFFFu, want)) {
        const float m_new = want ? mxs : m;
        // nothing to rescale while no row of the warp has seen a key
        if (__any_sync(0xFFFFFFFFu, m > -INFINITY)) {
            const float alpha = want ? ptx::ex2(m - m_new) : 1.0f;
            l *= alpha;
#pragma unroll
            for (int q = 0; q < HD / 32; ++q) {
                uint32_t o[32];
                ptx::tmem_ld32(tO + 32 * q, o);
                ptx::tmem_wait_ld();
                const uint64_t a2 = ptx::f2(alpha, alpha);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float x, y;
                    ptx::f2split(ptx::fmul2(ptx::f2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), a2), x, y);
                    o[e] = __float_as_uint(x);
                    o[e + 1] = __float_as_uint(y);
                }
                ptx::tmem_st32(tO + 32 * q, o);
            }
            ptx::tmem_wait_st();
        }
        m = m_new;
    }
    // upper key half first: its P V runs while the lower half is exponentiated
    uint32_t pk[32];
    l += exp64<kMask>(hi, valid - 64, c, m, pk);
    ptx::tmem_st32(tP + 32, *reinterpret_cast<uint32_t(*)[32]>(pk));
    ptx::tmem_wait_st();
    ptx::tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar_half);
    l += exp64<kMask>(lo, valid, c, m, pk);
    ptx::tmem_st32(tP, *reinterpret_cast<uint32_t(*)[32]>(pk));
    ptx::tmem_wait_st();
}

// What a CTA works on, from the device's lists; found by one warp.
struct Plan {
    int seq, row0, rows0, rows1, seen;   // rows of the two tiles, keys that any of them sees; rows0 = 0: nothing
};

// The x-th query tile pair of all sequences.  Later tiles of a sequence come
// first: under causal limits they see the most keys.
__device__ __forceinline__ Plan make_plan(const Args& a, int x, bool report) {
    const int lane = threadIdx.x & 31;
    const int step = 2 * a.tile_rows;
    Plan p{0, 0, 0, 0, 0};
    int done = 0;
    for (int s0 = 0; s0 < a.n_seqs; s0 += 32) {
        const int s = s0 + lane;
        int lo = 0, hi = 0, len = 0, tiles = 0;
        if (s < a.n_seqs) {
            lo = __ldg(a.cu + s);
            hi = __ldg(a.cu + s + 1);
            len = __ldg(a.lens + s);
            const bool ok = lo >= 0 && lo <= hi && hi <= a.n_rows && hi - lo <= a.max_rows && len >= 0 &&
                            len <= a.max_len && (s > 0 || lo == 0);
            if (!ok && report) raise_error(a.err, JANO_EINDEX);
            tiles = ok ? (hi - lo + step - 1) / step : 0;
        }
        int sum = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += v;
        }
        const bool mine = x >= done + sum - tiles && x < done + sum;
        const unsigned who = __ballot_sync(0xFFFFFFFFu, mine);
        if (who) {
            const int src = __ffs(who) - 1;
            const int t = tiles - 1 - (x - (done + sum - tiles));
            const int first = lo + t * step;
            p.seq = s0 + src;
            p.row0 = __shfl_sync(0xFFFFFFFFu, first, src);
            const int left = __shfl_sync(0xFFFFFFFFu, hi - first, src);
            p.rows0 = min(left, a.tile_rows);
            p.rows1 = min(left - p.rows0, a.tile_rows);
            p.seen = __shfl_sync(0xFFFFFFFFu, len, src);
            break;
        }
        done += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (a.limits && p.rows0 > 0) {
        int most = 0;
        for (int i = lane; i < p.rows0 + p.rows1; i += 32) most = max(most, __ldg(a.limits + p.row0 + i));
        p.seen = min(p.seen, __reduce_max_sync(0xFFFFFFFFu, most));
    }
    return p;
}

// Parts of a tile row: one per CTA of the cluster, two (the streams) in the
// single form.  With M the largest m and w = 2^(m - M),
//   out = sum w O / sum w l,   summed in a fixed order;
// one softmax warp per row, the rows dealt over the cluster's.  The plan is
// read again from shared memory, so nothing of it is held through the loops.
template <int HD>
__device__ __forceinline__ void merge_rows(const Args& a) {
    using L = Layout<HD>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const volatile int* plan = reinterpret_cast<const volatile int*>(smem_raw + (base - raw) + L::kMisc + 16);
    const int row0 = plan[1], rows0 = plan[2], rows1 = plan[3];
    const bool single = rows1 == 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_split = (int)gridDim.z;
    constexpr int E = HD / 32;                     // columns per lane
    const int packed0 = rows0 * a.group, total = packed0 + rows1 * a.group;
    const int parts = single ? 2 * n_split : n_split;
    for (int r = (int)blockIdx.z * kSoftmaxWarps + warp; r < total; r += n_split * kSoftmaxWarps) {
        const int tile = r >= packed0, p = tile ? r - packed0 : r;
        // lane = part: its address, weight and share of the sum
        const int z = single ? lane >> 1 : lane, st = single ? lane & 1 : tile;
        uint32_t row_addr = 0;
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < parts) {
            const uint32_t peer = ptx::mapa_shared(base, (uint32_t)z);
            ml = ld_cluster_f2(peer + L::kMl + (st * BM + p) * 8);
            row_addr = peer + (st * BM + p) * L::kRow * 4;
        }
        if (__any_sync(0xFFFFFFFFu, ml.y < 0.f)) continue;     // a part is missing: JANO_ETIMEOUT was raised
        float M = ml.x, sum;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
        // a part without visible keys has m = -inf, l = 0 and no O
        const float w = ml.y != 0.f ? ptx::ex2(ml.x - M) : 0.f;
        sum = w * ml.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        float acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
        for (int c = 0; c < parts; ++c) {
            const float wc = __shfl_sync(0xFFFFFFFFu, w, c);
            const uint32_t ac = __shfl_sync(0xFFFFFFFFu, row_addr, c);
            if (wc != 0.f) {
                if constexpr (E == 4) {
                    const float4 o = ld_cluster_f4(ac + lane * 16);
                    acc[0] = fmaf(wc, o.x, acc[0]);
                    acc[1] = fmaf(wc, o.y, acc[1]);
                    acc[2] = fmaf(wc, o.z, acc[2]);
                    acc[3] = fmaf(wc, o.w, acc[3]);
                } else {
                    const float2 o = ld_cluster_f2(ac + lane * 8);
                    acc[0] = fmaf(wc, o.x, acc[0]);
                    acc[1] = fmaf(wc, o.y, acc[1]);
                }
            }
        }
        const float inv = sum != 0.f ? 1.0f / sum : 0.f;
        __nv_bfloat16* dst = a.out + (long long)(row0 + tile * a.tile_rows + p / a.group) * a.out_ld +
                             ((int)blockIdx.y * a.group + p % a.group) * HD + lane * E;
        if constexpr (E == 4)
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(ptx::pack_bf16(acc[0] * inv, acc[1] * inv), ptx::pack_bf16(acc[2] * inv, acc[3] * inv));
        else
            *reinterpret_cast<uint32_t*>(dst) = ptx::pack_bf16(acc[0] * inv, acc[1] * inv);
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
    const int head = blockIdx.y;                       // K/V head
    const int n_split = (int)gridDim.z, split = (int)blockIdx.z;

    Ctl ctl;
    ctl.bar0 = base + L::kBar;
    ctl.abort = reinterpret_cast<volatile int*>(gbase + L::kMisc + 4);
    ctl.err = a.err;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::kMisc);
    int* plan_slot = reinterpret_cast<int*>(gbase + L::kMisc + 16);

    if (warp == 0) {
        const Plan p = make_plan(a, (int)blockIdx.x, blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0);
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
            ptx::mbar_init(ctl.bar(L::bFull + s), 1);
            ptx::mbar_init(ctl.bar(L::bEmpty + s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(ctl.bar(L::bSFull + s), 1);
            ptx::mbar_init(ctl.bar(L::bPFull + s), 4);
            ptx::mbar_init(ctl.bar(L::bPHalf + s), 4);
            ptx::mbar_init(ctl.bar(L::bOFull + s), 1);
        }
        ptx::mbar_init(ctl.bar(L::bLast), 1);
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
    const LoadOrder order{single, n};
    const bool ragged = n > 0 && kt0 + n == nt && seen % BN != 0;   // this CTA holds the ragged last tile
    const bool merge = rows0 > 0 && (single || n_split > 1);

    if (warp >= 8) {
      ptx::setmaxnreg_dec<kRegsIssue>();
      if (warp == 8 && n > 0) {
        // ------------------------------------------------------------ producer
        if (elect_one()) {
            const uint32_t q_bytes = (uint32_t)(a.tile_rows * a.group * 128 * L::kPanels);
            ptx::mbar_arrive_expect_tx(ctl.bar(L::bQFull), single ? q_bytes : 2 * q_bytes);
            for (int p = 0; p < L::kPanels; ++p) {
                ptx::tma_load_3d(base + p * kPanel, &tmQ, ctl.bar(L::bQFull), p * 64, head * a.group, row0);
                if (!single)
                    ptx::tma_load_3d(base + L::kQ1 + p * kPanel, &tmQ, ctl.bar(L::bQFull), p * 64, head * a.group,
                                     row0 + a.tile_rows);
            }
            const int shift = a.page_shift, page_rows = 1 << shift;
            const int box_rows = min(page_rows, BN);
            const int32_t* pages = a.table + (long long)seq * a.max_pages;
            // the page ids of a load are read right after the load before it
            // went out, so they arrive while its slot is still in use
            int ids[kMaxBoxes];
            auto read_ids = [&](int i) {
                bool is_v;
                const int key0 = (kt0 + order.tile(i, is_v)) * BN;
                const int boxes = (min(seen - key0, BN) + box_rows - 1) / box_rows;
#pragma unroll
                for (int b = 0; b < kMaxBoxes; ++b)
                    if (b < boxes) ids[b] = __ldg(pages + ((key0 + b * box_rows) >> shift));
            };
            read_ids(0);
            int issued = 0;
            for (int i = 0; i < 2 * n; ++i) {
                bool is_v;
                const int key0 = (kt0 + order.tile(i, is_v)) * BN;
                const int live = min(seen - key0, BN);
                const int boxes = (live + box_rows - 1) / box_rows;
                const int s = i % L::kSlots;
                if (!ctl.wait(L::bEmpty + s, ((i / L::kSlots) & 1) ^ 1)) break;
#ifdef JANO_INJECT_DROP_LOAD
                // failure-path test builds only: this tile is never issued, so
                // the MMA's bounded wait for it runs out (JANO_ETIMEOUT)
                if (i == JANO_INJECT_DROP_LOAD) continue;
#endif
                const uint32_t bar = ctl.bar(is_v && live < BN ? L::bLast : L::bFull + s);
                ptx::mbar_arrive_expect_tx(bar, (uint32_t)(boxes * box_rows * 128 * L::kPanels));
                const CUtensorMap* tm = is_v ? &tmV : &tmK;
                const uint32_t dst = base + L::kRing + s * L::kTile;
#pragma unroll
                for (int b = 0; b < kMaxBoxes; ++b)
                    if (b < boxes) {
                        int page = ids[b];
                        if (page < 0 || page >= a.n_pages) {
                            raise_error(a.err, JANO_EINDEX);
                            page = a.n_pages;          // out of range: the copy fills zeros
                        }
                        for (int p = 0; p < L::kPanels; ++p)
                            tma_load_4d(dst + b * box_rows * 128 + p * kPanel, tm, bar, p * 64,
                                        key0 & (page_rows - 1), head, page);
                    }
                issued = i + 1;
                if (issued < 2 * n) read_ids(issued);
            }
            // drain: every copy this CTA issued lands before its smem is released
            ptx::mbar_wait(ctl.bar(L::bQFull), 0, kWaitLimit);
            for (int i = max(0, issued - L::kSlots); i < issued; ++i) {
#ifdef JANO_INJECT_DROP_LOAD
                if (i == JANO_INJECT_DROP_LOAD) continue;
#endif
                bool is_v;
                const int g = order.tile(i, is_v);
                if (is_v && seen - (kt0 + g) * BN < BN) ptx::mbar_wait(ctl.bar(L::bLast), 0, kWaitLimit);
                else ptx::mbar_wait(ctl.bar(L::bFull + i % L::kSlots), (i / L::kSlots) & 1, kWaitLimit);
            }
        }
      } else if (warp == 9 && n > 0) {
        // ------------------------------------------------------------ MMA issuer
        if (elect_one()) {
            constexpr uint32_t idesc_qk = ptx::idesc_bf16(BM, BN, false, false);
            constexpr uint32_t idesc_pv = ptx::idesc_bf16(BM, HD, false, true);
            auto slot_of = [](int i) { return i % L::kSlots; };
            auto wait_full = [&](int i) { return ctl.poll(L::bFull + slot_of(i), (i / L::kSlots) & 1); };
            auto release = [&](int i) { ptx::mma_commit(ctl.bar(L::bEmpty + slot_of(i))); };
            auto qk = [&](int st, uint32_t qb, int i) {    // S_st = Q K^T, K in load i's slot
                const uint32_t kd = desc_lo(base + L::kRing + slot_of(i) * L::kTile, 16), qd = desc_lo(qb, 16);
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * kPanel + (kk & 3) * 32) >> 4;
                    mma_ss(tmem + L::tS(st), qd + off, kd + off, idesc_qk, kk > 0);
                }
                ptx::mma_commit(ctl.bar(L::bSFull + st));
            };
            // O_st += P_st V over key sixteenths [k0, k1); V in load i's slot
            auto pv = [&](int st, int i, int k0, int k1, bool acc) {
                const uint32_t vd = desc_lo(base + L::kRing + slot_of(i) * L::kTile, kPanel);
#pragma unroll
                for (int kk = k0; kk < k1; ++kk)
                    mma_ts(tmem + L::tO(st), tmem + L::tS(st) + L::tP + kk * 8, vd + kk * 128, idesc_pv,
                           acc || kk > k0);
            };
            auto pv_tile = [&](int st, int i, int j) -> bool {
                if (!ctl.poll(L::bPHalf + st, j & 1)) return false;
                ptx::tc_fence_after();
                pv(st, i, BN / 32, BN / 16, j > 0);
                if (!ctl.poll(L::bPFull + st, j & 1)) return false;
                ptx::tc_fence_after();
                pv(st, i, 0, BN / 32, true);
                return true;
            };
            bool ok = ctl.poll(L::bQFull, 0);
            if (!single) {
                // S0_0 S1_0 | PV0_{j-1} S0_j PV1_{j-1} S1_j | ... PV0 PV1
                // (loads: K_j is 2j, V_j is 2j + 1)
                if (ok && (ok = wait_full(0))) {
                    ptx::tc_fence_after();
                    qk(0, base, 0);
                    qk(1, base + L::kQ1, 0);
                    release(0);
                }
                for (int j = 1; ok && j < n; ++j) {
                    const int ik = 2 * j, iv = 2 * j - 1;
                    if (!wait_full(iv) || !wait_full(ik)) { ok = false; break; }
                    if (!pv_tile(0, iv, j - 1)) { ok = false; break; }
                    qk(0, base, ik);
                    if (!pv_tile(1, iv, j - 1)) { ok = false; break; }
                    release(iv);
                    qk(1, base + L::kQ1, ik);
                    release(ik);
                }
                if (ok) {
                    const int iv = 2 * n - 1;
                    ok = wait_full(iv) && pv_tile(0, iv, n - 1);
                    if (ok) {
                        ptx::mma_commit(ctl.bar(L::bOFull + 0));
                        ok = pv_tile(1, iv, n - 1);
                    }
                    if (ok) {
                        ptx::mma_commit(ctl.bar(L::bOFull + 1));
                        release(iv);
                    }
                }
            } else {
                // S0(0) S1(1) | PV(g) S(g+2) ... over the tiles g, stream g & 1
                const LoadOrder order{true, n};
                for (int g = -2; ok && g < n; g += 2) {
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        const int v = g + st, k = g + st + 2;
                        if (v >= 0 && v < n) {
                            if (!wait_full(order.v(v)) || !pv_tile(st, order.v(v), v >> 1)) { ok = false; break; }
                            release(order.v(v));
                            if (k >= n) ptx::mma_commit(ctl.bar(L::bOFull + st));
                        }
                        if (k < n) {
                            if (!wait_full(order.k(k))) { ok = false; break; }
                            ptx::tc_fence_after();
                            qk(st, base, order.k(k));
                            release(order.k(k));
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
        const int i = order.v(n - 1);
        if (ctl.warp_wait(L::bLast, 0)) {
            const int live = seen - (nt - 1) * BN;
            uint8_t* v = gbase + L::kRing + (i % L::kSlots) * L::kTile;
            for (int e = live * 8 + lane; e < BN * 8; e += 32)
                for (int p = 0; p < L::kPanels; ++p)
                    *reinterpret_cast<uint4*>(v + p * kPanel + e * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async();           // ordered before the tensor core's reads
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ctl.bar(L::bFull + i % L::kSlots));
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
        const uint32_t tS = tmem + lane_off + L::tS(i);
        const uint32_t tO = tmem + lane_off + L::tO(i);
        const bool warp_live = q * 32 < (i && !single ? rows1 : rows0) * a.group;   // else only the barriers are kept
        const int steps = single ? (n + 1 - i) >> 1 : n;
        // the stream's tiles start at keys first, first + apart, ...
        const int first = (kt0 + (single ? i : 0)) * BN, apart = single ? 2 * BN : BN;
        int limit = seen;
        if (a.limits && row < (i && !single ? rows1 : rows0) * a.group)
            limit = min(seen, __ldg(a.limits + row0 + (i && !single ? a.tile_rows : 0) + row / a.group));
        // steps whose tile every row of the warp sees whole; the rest is masked
        const int whole = __reduce_min_sync(0xFFFFFFFFu, limit) - first - BN;
        const int plain = whole < 0 ? 0 : min(steps, whole / apart + 1);
        float m = -INFINITY, l = 0.f;
        int j = 0;
        if (warp_live) {
            for (; j < plain; ++j) {
                if (!ctl.warp_wait(L::bSFull + i, j & 1)) break;
                ptx::tc_fence_after();
                softmax_tile<HD, false>(tS, BN, a.scale_log2, m, l, ctl.bar(L::bPHalf + i));
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ctl.bar(L::bPFull + i));
            }
            for (; j < steps; ++j) {
                if (!ctl.warp_wait(L::bSFull + i, j & 1)) break;
                ptx::tc_fence_after();
                softmax_tile<HD, true>(tS, limit - first - j * apart, a.scale_log2, m, l, ctl.bar(L::bPHalf + i));
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

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

bool encode(CUtensorMap* m, const void* ptr, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(ptr), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows [n_rows][heads][d]: a box is one tile's query rows x the heads of a group x 64 columns.
bool make_q_map(CUtensorMap* m, const void* q, long long ld, int n_rows, int heads, int d, int group, int tile_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)n_rows};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)tile_rows};
    return encode(m, q, 3, dims, strides, box);
}

// The pool [page][place][head][d] with its own strides: a box is up to 128 places of one page and head x 64 columns.
bool make_pool_map(CUtensorMap* m, const void* pages, const jano_page_pool& p) {
    const cuuint64_t dims[4] = {(cuuint64_t)p.d, (cuuint64_t)p.page_size, (cuuint64_t)p.kv_heads,
                                (cuuint64_t)p.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)p.token_stride * 2, (cuuint64_t)p.head_stride * 2,
                                   (cuuint64_t)p.page_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)(p.page_size < BN ? p.page_size : BN), 1, 1};
    return encode(m, pages, 4, dims, strides, box);
}

template <int HD>
cudaError_t set_up(int dev, int& max_cluster) {
    using L = Layout<HD>;
    static DeviceOnce ready;
    static std::atomic<int> cluster_of[64];
    if (!ready.done(dev)) {
        // the register split assumes exactly kRegsLaunch registers per thread
        cudaFuncAttributes fa;
        cudaError_t e = cudaFuncGetAttributes(&fa, paged_attention_kernel<HD>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
        e = cudaFuncSetAttribute(paged_attention_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)L::kAlloc);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(paged_attention_kernel<HD>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        // clusters of 16 CTAs need 16 free SMs in one GPC: asked once per device
        cudaLaunchConfig_t cfg{};
        cudaLaunchAttribute attr[1];
        cfg.gridDim = dim3(1, 1, 16);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = L::kAlloc;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {1, 1, 16};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int active = 0;
        const bool wide = cudaOccupancyMaxActiveClusters(&active, paged_attention_kernel<HD>, &cfg) == cudaSuccess &&
                          active > 0;
        if (!wide) cudaGetLastError();
        if (dev >= 0 && dev < 64) cluster_of[dev].store(wide ? 16 : 8, std::memory_order_relaxed);
        ready.mark(dev);
        max_cluster = wide ? 16 : 8;
        return cudaSuccess;
    }
    max_cluster = cluster_of[dev].load(std::memory_order_relaxed);
    return cudaSuccess;
}

template <int HD>
cudaError_t launch_hd(const PagedAttentionCall& c, const Args& a, int tiles, int* err, cudaStream_t st) {
    using L = Layout<HD>;
    int dev = 0, max_cluster = 8;
    cudaGetDevice(&dev);
    cudaError_t e = set_up<HD>(dev, max_cluster);
    if (e != cudaSuccess) return e;
    int sms = 148;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    int split = c.n_split;
    if (split == 0)
        split = paged_split_count(c.n_rows, c.max_rows, c.max_len, c.seqs->n_seqs, c.heads, c.pool->kv_heads, sms);
    if (split > max_cluster) split = max_cluster;
    CUtensorMap mq, mk, mv;
    if (!make_q_map(&mq, c.q, c.q_ld, c.n_rows, c.heads, HD, a.group, a.tile_rows) ||
        !make_pool_map(&mk, c.pool->k, *c.pool) || !make_pool_map(&mv, c.pool->v, *c.pool))
        return cudaErrorInvalidValue;
    const dim3 grid((unsigned)tiles, (unsigned)c.pool->kv_heads, (unsigned)split);
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

// CTAs per (query tile pair, K/V head): the cluster size z (1, 2, 4, 8, 16)
// with the shortest modelled time, rounds of z C CTAs over the SMs times the
// key tiles of one CTA plus the equivalent of `fixed` tiles for its set-up,
// pipeline fill and merge.
int paged_split_count(int n_rows, int max_rows, int max_len, int n_seqs, int heads, int kv_heads, int sms) {
    if (n_rows <= 0 || max_rows <= 0 || max_len <= 0 || sms <= 0) return 1;
    const int tile_rows = BM / (heads / kv_heads);
    const double ctas = (double)tile_bound(n_rows, max_rows, n_seqs, tile_rows) * kv_heads;
    const int nt = (max_len + BN - 1) / BN;
    const double fixed = 12.0;
    int best = 1;
    double best_t = 0.0;
    for (int z = 1; z <= kMaxSplit && (z == 1 || nt >= 2 * z); z *= 2) {
        const double w = ctas * z / sms;
        const double full = std::floor(w), f = w - full;
        const double rounds = full + (f > 1e-9 ? 0.7 + 0.3 * f : 0.0);
        const double t = rounds * ((double)nt / z + fixed);
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
    return c.pool->d == 128 ? launch_hd<128>(c, a, (int)tiles, err, st) : launch_hd<64>(c, a, (int)tiles, err, st);
}

}  // namespace jano
