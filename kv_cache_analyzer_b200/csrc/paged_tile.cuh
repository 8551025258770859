// paged_tile.cuh -- what the two paged attention kernels share: bounded waits,
// single-thread issue of the tensor core's instructions, the order of the K/V
// loads, the softmax of one key tile, and the tensor maps of rows and pools.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "jano_common.cuh"

namespace jano {
namespace {

constexpr int BM = 128;                      // rows of an MMA tile
constexpr int BN = 128;                      // keys per tile
constexpr uint32_t kPanel = 128 * 128;       // bytes of one 128-row x 64-column panel
#ifndef JANO_WAIT_CYCLES
#define JANO_WAIT_CYCLES (1ll << 31)         // (test builds: shorter)
#endif
constexpr long long kWaitLimit = JANO_WAIT_CYCLES;   // ~1 s
// A wait that spans key tiles, not the step of one: some more for each.  (A
// tile takes up to 4,100 cycles, 2^26 keys in one CTA 1.1 s; where something
// else failed, the abort flag ends the wait.)
__device__ __forceinline__ long long span_limit(int tiles) { return kWaitLimit + (long long)tiles * 16384; }

// Tensor memory of the two streams: S0 [0,128) S1 [128,256) O0 [256,256+d)
// O1 [384,384+d); P_i, BF16, over the upper half of S_i.
__host__ __device__ constexpr uint32_t tmem_s(int i) { return i ? 128u : 0u; }
__host__ __device__ constexpr uint32_t tmem_o(int i) { return i ? 384u : 256u; }
constexpr uint32_t kTmemP = 64;
static_assert(tmem_o(1) - tmem_s(1) == tmem_o(0) - tmem_s(0), "O lies at one distance from S");

struct Ctl {
    uint32_t bar0;
    volatile int* abort;
    int* err;
    __device__ uint32_t bar(int i) const { return bar0 + 8u * (uint32_t)i; }
    // Waiting threads sleep until the phase completes; the MMA warp polls
    // (its waits sit on every key tile's critical path).
    __device__ bool wait(int i, uint32_t parity, long long limit = kWaitLimit) const {
        if (ptx::mbar_try_wait_sleep(bar(i), parity)) return true;
        const long long t0 = clock64();
        for (;;) {
            if (ptx::mbar_try_wait_sleep(bar(i), parity)) return true;
            if (*abort) return false;
            if (clock64() - t0 > limit) {
                *abort = 1;
                raise_error(err, JANO_ETIMEOUT);
                return false;
            }
        }
    }
    __device__ bool poll(int i, uint32_t parity, long long limit = kWaitLimit) const {
        if (ptx::mbar_try_wait(bar(i), parity)) return true;
        const long long t0 = clock64();
        while (!ptx::mbar_try_wait(bar(i), parity)) {
            if (*abort) return false;
            if (clock64() - t0 > limit) {
                *abort = 1;
                raise_error(err, JANO_ETIMEOUT);
                return false;
            }
        }
        return true;
    }
    // Warp-uniform: the .sync.aligned operations that follow never diverge.
    __device__ bool warp_wait(int i, uint32_t parity, long long limit = kWaitLimit) const {
        int ok = 0;
        if ((threadIdx.x & 31) == 0) ok = wait(i, parity, limit) ? 1 : 0;
        return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
    }
    __device__ bool warp_poll(int i, uint32_t parity, long long limit = kWaitLimit) const {
        int ok = 0;
        if ((threadIdx.x & 31) == 0) ok = poll(i, parity, limit) ? 1 : 0;
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

// The ring of K or of V tiles in shared memory, as its producer or its consumer
// counts through it.
struct RingPos {
    int slots;
    int slot = 0, phase = 0;
    __device__ __forceinline__ explicit RingPos(int n) : slots(n) {}
    __device__ __forceinline__ void advance() {
        if (++slot == slots) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// One thread's feed of one operand (K or V) into its ring of tiles, by
// page-sized copies.  K and V have a producer each: a lone thread runs some
// five cycles per instruction, and one producer for both took 1,300 cycles per
// 32 KB tile (page ids, bounds, barrier, coordinates), as long as the copy.
template <int HD, bool kSpin>
struct Feed {
    static constexpr int kPanels = HD / 64;
    const Ctl& ctl;
    const CUtensorMap* map;
    int b_full, b_empty, b_land;       // barriers; the ragged last V tile lands on b_land (K: b_full) ...
    bool is_v;                         // ... and is cleared past its last key before b_full
    uint32_t ring;
    RingPos pos;
    uint32_t landing = 0, land_phase = 0;      // by slot: last load went to b_land; parity of its next phase
    int loads = 0;

    // NB pages a tile.  Key tiles [kt0, kt0 + n) of the sequence whose page ids
    // are `pages`, its keys from `seen` on left out; false: a wait gave up.
    template <int NB>
    __device__ __forceinline__ bool run(const int32_t* pages, int shift, int n_pages, int kt0, int n, int seen,
                                        int head) {
        const int rows = NB == 1 ? BN : 1 << shift;    // keys per copy
        const int place_mask = (1 << shift) - 1;
        int ids[NB];
        auto read_ids = [&](int key0) {
            const int first = key0 >> shift;
#pragma unroll
            for (int b = 0; b < NB; ++b)
                if (b == 0 || key0 + b * rows < seen) ids[b] = key0 < seen ? __ldg(pages + first + b) : 0;
        };
        int key0 = kt0 * BN;
        read_ids(key0);
        for (int g = 0; g < n; ++g, key0 += BN) {
            const int live = min(seen - key0, BN);
            const int boxes = NB == 1 ? (live > 0 ? 1 : 0) : (live + rows - 1) >> shift;
            if (!(kSpin ? ctl.poll(b_empty + pos.slot, pos.phase ^ 1) : ctl.wait(b_empty + pos.slot, pos.phase ^ 1)))
                return false;
#ifdef JANO_INJECT_DROP_LOAD
            // failure-path test builds only: one K tile is never issued, so the
            // MMA's bounded wait for it runs out (JANO_ETIMEOUT)
            if (!is_v && loads == JANO_INJECT_DROP_LOAD) return false;
#endif
            const bool land = is_v && live < BN;
            const uint32_t bar = ctl.bar((land ? b_land : b_full) + pos.slot);
            landing = (landing & ~(1u << pos.slot)) | ((land ? 1u : 0u) << pos.slot);
            if (land) land_phase ^= 1u << pos.slot;
            ptx::mbar_arrive_expect_tx(bar, (uint32_t)(boxes * rows * 128 * kPanels));
            const uint32_t dst = ring + pos.slot * kPanels * kPanel;
#pragma unroll
            for (int b = 0; b < NB; ++b)
                if (b < boxes) {
                    int page = ids[b];
                    if ((unsigned)page >= (unsigned)n_pages) {
                        raise_error(ctl.err, JANO_EINDEX);
                        page = n_pages;                // out of range: the copy fills zeros
                    }
#pragma unroll
                    for (int p = 0; p < kPanels; ++p)
                        tma_load_4d(dst + b * rows * 128 + p * kPanel, map, bar, p * 64, key0 & place_mask, head, page);
                }
            ++loads;
            pos.advance();
            // the next tile's page ids arrive while its slot is still in use
            if (g + 1 < n) read_ids(key0 + BN);
        }
        return true;
    }
    __device__ __forceinline__ bool tiles(const int32_t* pages, int shift, int n_pages, int kt0, int n, int seen,
                                          int head) {
        if (shift >= 7) return run<1>(pages, shift, n_pages, kt0, n, seen, head);
        if (shift == 6) return run<2>(pages, shift, n_pages, kt0, n, seen, head);
        if (shift == 5) return run<4>(pages, shift, n_pages, kt0, n, seen, head);
        return run<8>(pages, shift, n_pages, kt0, n, seen, head);
    }
    // Every copy that was issued lands before the CTA's shared memory is released.
    __device__ __forceinline__ void drain() {
        for (int k = 0; k < pos.slots; ++k) {
            const int before = loads - 1 - k;          // loads counted back from the last
            if (before < 0) break;
            const int at = before % pos.slots;
            const bool land = (landing >> at) & 1u;
            if (!ptx::mbar_wait(ctl.bar((land ? b_land : b_full) + at),
                                land ? ((land_phase >> at) & 1u) ^ 1u : (before / pos.slots) & 1, kWaitLimit))
                break;
        }
    }
};

// Row max of 64 values (8 independent chains of 3-input max).
__device__ __forceinline__ float max64(const uint32_t (&s)[64]) {
    float m[8];
#pragma unroll
    for (int a = 0; a < 8; ++a) m[a] = -INFINITY;
#pragma unroll
    for (int e = 0; e < 64; e += 2)
        m[(e >> 1) & 7] = ptx::fmax3(m[(e >> 1) & 7], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
    return fmaxf(ptx::fmax3(m[0], m[1], m[2]), ptx::fmax3(m[3], m[4], fmaxf(m[5], fmaxf(m[6], m[7]))));
}

// 2^x for two lanes on the FMA and ALU pipes, for x <= 8: the range reduction
// and the cubic of attention.cu (largest relative error 7.5e-5, below the 2^-8
// rounding of the BF16 P it feeds).
__device__ __forceinline__ void exp2_poly2(uint64_t x2, float& ya, float& yb) {
    constexpr float kC0 = 0x1.fff692p-1f, kC1 = 0x1.62f31ap-1f;
    constexpr float kC2 = 0x1.f0de1ap-3f, kC3 = 0x1.c3f76p-5f;
    constexpr float kRound = 12582912.0f;            // 1.5 * 2^23
    float xa, xb;
    ptx::f2split(x2, xa, xb);
    x2 = ptx::f2(fmaxf(xa, -125.0f), fmaxf(xb, -125.0f));
    const uint64_t r2 = ptx::fadd2(x2, ptx::f2(kRound, kRound));     // low bits hold rint(x)
    const uint64_t t2 = ptx::fadd2(r2, ptx::f2(-kRound, -kRound));
    const uint64_t f2 = ptx::ffma2(t2, ptx::f2(-1.f, -1.f), x2);      // f = x - rint(x)
    uint64_t p2 = ptx::ffma2(ptx::f2(kC3, kC3), f2, ptx::f2(kC2, kC2));
    p2 = ptx::ffma2(p2, f2, ptx::f2(kC1, kC1));
    p2 = ptx::ffma2(p2, f2, ptx::f2(kC0, kC0));
    float ra, rb, pa, pb;
    ptx::f2split(r2, ra, rb);
    ptx::f2split(p2, pa, pb);
    const int ja = __float_as_int(ra) - __float_as_int(kRound);
    const int jb = __float_as_int(rb) - __float_as_int(kRound);
    ya = __int_as_float(__float_as_int(pa) + (ja << 23));
    yb = __int_as_float(__float_as_int(pb) + (jb << 23));
}

// p = 2^(s*c + nm) for 64 values, packed to 32 BF16x2 words; returns sum(p).
// kPoly of 8 pairs go through exp2_poly2.
template <int kPoly>
__device__ __forceinline__ float exp64(const uint32_t (&s)[64], float c, float nm, uint32_t* pk) {
    const uint64_t c2 = ptx::f2(c, c), nm2 = ptx::f2(nm, nm);
    uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
    for (int e = 0; e < 64; e += 2) {
        const uint64_t x2 = ptx::ffma2(ptx::f2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, nm2);
        float a, b;
        if (((e >> 1) & 7) < kPoly) {
            exp2_poly2(x2, a, b);
        } else {
            ptx::f2split(x2, a, b);
            a = ptx::ex2(a);
            b = ptx::ex2(b);
        }
        acc[(e >> 1) & 3] = ptx::fadd2(acc[(e >> 1) & 3], ptx::f2(a, b));
        pk[e >> 1] = ptx::pack_bf16(a, b);
    }
    float lo, hi;
    ptx::f2split(ptx::fadd2(ptx::fadd2(acc[0], acc[1]), ptx::fadd2(acc[2], acc[3])), lo, hi);
    return lo + hi;
}

// One key tile of one tile row (see the file comments): S from TMEM, maximum,
// lazy rescale of O, P back as BF16.  With `masked` (the same in the whole
// warp) the row sees the tile's first `valid` keys only: the other logits
// become -inf, whatever S holds there, and their P exactly 0.  The decode form
// passes it at run time: there a second copy would cost each CTA the
// instruction fetch of 20 KB at its last tile.
//
// kPoly: share of the exponentials, in eighths, kept off the MUFU unit.  A tile
// of 2 x 128 rows keeps it busy for 2,048 cycles and the tensor core for 1,024
// with d = 64, twice that with d = 128: 4,096 rows over 16,384 keys of 24 heads
// of 64 take 689, 676, 635, 609, 645 us with 0 to 4 eighths, of 128 alike from
// 0 to 3 (750 to 800, the power limit).  One warp per stream, as in the decode
// form, gains nothing (96.2 us of a batch with 0, 96.6 with 2, 103.9 with 3).
// A masked tile's P must be exactly 0, which the polynomial never is.
template <int HD, int kPoly>
__device__ __forceinline__ void softmax_tile(uint32_t tS, bool masked, int valid, float c, float& m, float& l,
                                             uint32_t bar_half) {
    const uint32_t tO = tS + (tmem_o(0) - tmem_s(0)), tP = tS + kTmemP;
    uint32_t s[128];
    ptx::tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
    ptx::tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
    ptx::tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&s[64]));
    ptx::tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&s[96]));
    ptx::tmem_wait_ld();
    if (masked) {
#pragma unroll
        for (int e = 0; e < 128; ++e)
            if (e >= valid) s[e] = 0xFF800000u;
    }
    const uint32_t(&lo)[64] = *reinterpret_cast<const uint32_t(*)[64]>(&s[0]);
    const uint32_t(&hi)[64] = *reinterpret_cast<const uint32_t(*)[64]>(&s[64]);
    const float mxs = fmaxf(max64(lo), max64(hi)) * c;
    const bool want = mxs > m + 8.0f;
    if (__any_sync(0xFFFFFFFFu, want)) {
        const float m_new = want ? mxs : m;
        // nothing to rescale while no row of the warp has seen a key (m = -inf;
        // a lane without a row has m = inf)
        if (__any_sync(0xFFFFFFFFu, fabsf(m) < INFINITY)) {
            const float alpha = want ? ptx::ex2(m - m_new) : 1.0f;
            l *= alpha;
#pragma unroll 1
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
    // a row that has seen no key yet has m = -inf and only masked logits: P = 0
    const float nm = m > -INFINITY ? -m : 0.0f;
    // upper key half first: its P V runs while the lower half is exponentiated
    uint32_t pk[32];
    l += exp64<kPoly>(hi, c, nm, pk);
    ptx::tmem_st32(tP + 32, *reinterpret_cast<uint32_t(*)[32]>(pk));
    ptx::tmem_wait_st();
    ptx::tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar_half);
    l += exp64<kPoly>(lo, c, nm, pk);
    ptx::tmem_st32(tP, *reinterpret_cast<uint32_t(*)[32]>(pk));
    ptx::tmem_wait_st();
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
            const cuuint32_t* box, CUtensorMapL2promotion fetch) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(ptr), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, fetch,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows [n_rows][heads][d]: a box is one tile's query rows x the heads of a group x 64 columns.
bool make_q_map(CUtensorMap* m, const void* q, long long ld, int n_rows, int heads, int d, int group, int tile_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)n_rows};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)tile_rows};
    return encode(m, q, 3, dims, strides, box, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// The pool [page][place][head][d] with its own strides: a box is up to 128 places of one page and head x 64 columns.
bool make_pool_map(CUtensorMap* m, const void* pages, const jano_page_pool& p) {
    const cuuint64_t dims[4] = {(cuuint64_t)p.d, (cuuint64_t)p.page_size, (cuuint64_t)p.kv_heads,
                                (cuuint64_t)p.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)p.token_stride * 2, (cuuint64_t)p.head_stride * 2,
                                   (cuuint64_t)p.page_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)(p.page_size < BN ? p.page_size : BN), 1, 1};
    // L2 fetches a head's row at once, and not its neighbour's: with 256 bytes
    // for d = 64, 32 sequences of 8,192 tokens (token-major) took 139 us, not 100
    return encode(m, pages, 4, dims, strides, box,
                  p.d == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

}  // namespace
}  // namespace jano
