// rope.cu -- rotary positions with several axes (frame, row, column), alone
// and on the way into the KV cache: the token-ordered one or a page pool.
//
// A head's first `rot` columns form rot/2 slots, each a pair of columns; slot
// s belongs to one axis and turns its pair by the angle of the token's
// coordinate on that axis (cos and sin come from a table made once per
// geometry, in fp64, by the kernel below):
//   (x0, x1) -> (x0 c - x1 s, x0 s + x1 c),
// in fp32 with one rounding to BF16; columns past rot are moved bit for bit.
//
// Every row is read once and written once: bound by HBM, and close behind by
// the issue of instructions, so addresses go up by constants and the pairs are
// turned two at a time.  One warp takes one row (or, when there are too few
// rows to fill the SMs, a part of one) of one of up to three tensors (q, k, v:
// one launch for all), resolves the row's place and coordinates once, and
// walks its heads 32 units at a time.  A unit is the 16-byte vector of 4
// adjacent pairs (interleaved pairing) or the two vectors that hold 8 split
// pairs (halves pairing), so a pair never crosses lanes.  Where the units of a
// head divide 32 (d = 64 and 128 rotated whole, among others) a lane meets the
// same slots in every head and keeps its cos and sin in registers for the
// whole row.
//
// 18,900 rows of 40 heads of 128 (387 MB): 61.5 us, 6.3 TB/s; Q, K and V of
// 11,466 rows of 12 heads of 128 into the cache (211 MB): 35.6 us, 5.9 TB/s,
// as many into pages 38.1 us; a few rows: 2.2 us, the launch.
#include <cuda_bf16.h>

#include "jano_common.cuh"

namespace jano {
namespace {

constexpr int kWarps = 4;

struct Tab {
    const float2* cs;                      // [n_pos0][ns0], [n_pos1][ns1], [n_pos2][ns2]
    int ns[3];                             // slots per axis
    int np[3];                             // positions per axis
    int slots;                             // ns0 + ns1 + ns2
};

// Which token a row is, from where its coordinates come, and where its cache
// row lies (in 16-byte vectors).
struct Place {
    const int32_t* ids;                    // token id / cache position of row r (NULL: r)
    const int32_t* coords;                 // [n_rows][3] or NULL (from the id and the grid)
    const int32_t* grids;                  // [n_seqs][2] (rows, columns) or NULL
    int grid_h, grid_w;
    int ascending;                         // ids must rise strictly (within a sequence)
    int n_tokens;                          // bound of the ids; contiguous cache only
    // page pool (table NULL: contiguous or no cache)
    const int32_t* table;
    const int32_t* lens;
    const int32_t* cu;
    int n_seqs, max_pages, n_pages, page_shift;
    long long page_stride, token_stride, head_stride;
};

struct Job {
    const uint4* src;
    uint4* dst;
    long long src_ld, dst_ld;              // vectors between rows (dst_ld: direct rows only)
    long long dst_head;                    // vectors between heads of dst
    int heads;
    int rotate;
    int cached;                            // dst is the cache
};

struct Args {
    Job job[3];
    int n_jobs, n_rows, parts, d_vec;
    Tab tab;
    Place at;
    int* err;
};

// Sequence of row r: the s with cu[s] <= r < cu[s+1], by a 32-ary search of
// the whole warp; -1 if the row belongs to none (rows behind the last
// sequence), -2 if cu is not an ascending list from 0.
__device__ __forceinline__ int seq_of_row(const int32_t* cu, int n_seqs, int r) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = n_seqs;                // candidates [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;    // lane's candidate block starts here
        const bool before = lane * step < n && __ldg(cu + i) <= r;
        const int c = __popc(__ballot_sync(0xFFFFFFFFu, before));
        if (c == 0) break;
        const int first = lo + (c - 1) * step;
        n = min(step, lo + n - first);
        lo = first;
        if (step == 1) break;
    }
    const int a = __ldg(cu + lo), b = __ldg(cu + lo + 1);
    // (a sequence that begins at 0 behind others: these must be without rows)
    if (a <= r && r < b) return a > 0 ? (lo > 0 ? lo : -2) : (a == 0 && (lo == 0 || __ldg(cu) == 0) ? lo : -2);
    // behind the last sequence: the search ends there, and it ends before r
    return lo == n_seqs - 1 && a <= b && b <= r && __ldg(cu) == 0 ? -1 : -2;
}

// Coordinates, cache base and validity of a row; false: the row is skipped.
// The same for each of a row's tensors, those that are not rotated among them:
// a row is written whole or not at all.
__device__ __forceinline__ bool resolve(const Args& a, int r, int t, int t_before, int (&p)[3], long long& base) {
    const Place& w = a.at;
    int seq = 0;
    int first = 0;
    if (w.table) {
        seq = seq_of_row(w.cu, w.n_seqs, r);
        if (seq == -1) return false;
        if (seq < 0) { raise_error(a.err, JANO_EINDEX); return false; }
        first = __ldg(w.cu + seq);
    }
    bool bad = t < 0 || (w.ascending && r > first && t_before >= t);
    base = 0;
    if (w.table) {
        const int page_i = t >> w.page_shift;
        bad = bad || t >= __ldg(w.lens + seq) || page_i >= w.max_pages;
        if (!bad) {
            const int page = __ldg(w.table + (long long)seq * w.max_pages + page_i);
            bad = page < 0 || page >= w.n_pages;
            base = (long long)page * w.page_stride + (long long)(t & ((1 << w.page_shift) - 1)) * w.token_stride;
        }
    } else if (w.n_tokens) {
        bad = bad || t >= w.n_tokens;
        base = (long long)t * w.token_stride;
    }
    if (!bad && a.tab.slots > 0) {                         // (0: a call without a rotation)
        if (w.coords) {
            p[0] = __ldg(w.coords + 3ll * r);
            p[1] = __ldg(w.coords + 3ll * r + 1);
            p[2] = __ldg(w.coords + 3ll * r + 2);
        } else {
            const int gh = w.grids ? __ldg(w.grids + 2 * seq) : w.grid_h;
            const int gw = w.grids ? __ldg(w.grids + 2 * seq + 1) : w.grid_w;
            bad = gh < 1 || gw < 1;
            if (!bad) {
                const int row = t / gw;
                p[0] = row / gh;
                p[1] = row % gh;
                p[2] = t % gw;
            }
        }
#pragma unroll
        for (int x = 0; x < 3; ++x)
            bad = bad || (a.tab.ns[x] > 0 && (p[x] < 0 || p[x] >= a.tab.np[x]));
    }
    if (bad) raise_error(a.err, JANO_EINDEX);
    return !bad;
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// cos and sin of N slots from `slot` on; (1, 0) past the last one.
template <int N>
__device__ __forceinline__ void load_cs(const Tab& t, const int (&p)[3], int slot, float (&c)[N], float (&s)[N]) {
    const int b0 = p[0] * t.ns[0];
    const int b1 = t.np[0] * t.ns[0] + p[1] * t.ns[1] - t.ns[0];
    const int b2 = t.np[0] * t.ns[0] + t.np[1] * t.ns[1] + p[2] * t.ns[2] - t.ns[0] - t.ns[1];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int q = slot + i;
        const int b = q < t.ns[0] ? b0 : (q < t.ns[0] + t.ns[1] ? b1 : b2);
        float2 v = make_float2(1.f, 0.f);
        if (q < t.slots) v = __ldg(t.cs + b + q);
        c[i] = v.x;
        s[i] = v.y;
    }
}

// The 4 adjacent pairs of a vector, two at a time in packed fp32; pairs from
// slot `live` on are kept.  (The issue of instructions counts next to the
// bytes here: 35.1 us for the Q, K and V of 11,466 rows, 36.9 pair by pair.)
__device__ __forceinline__ uint4 turn_pairs(uint4 x, const float (&c)[4], const float (&s)[4], int live) {
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const uint64_t x0 = ptx::f2(lo_f(w[i]), lo_f(w[i + 1])), x1 = ptx::f2(hi_f(w[i]), hi_f(w[i + 1]));
        const uint64_t cc = ptx::f2(c[i], c[i + 1]), ss = ptx::f2(s[i], s[i + 1]);
        float a0, b0, a1, b1;
        ptx::f2split(ptx::ffma2(x0, cc, ptx::fmul2(x1, ptx::f2(-s[i], -s[i + 1]))), a0, b0);
        ptx::f2split(ptx::ffma2(x0, ss, ptx::fmul2(x1, cc)), a1, b1);
        const uint32_t ya = ptx::pack_bf16(a0, a1), yb = ptx::pack_bf16(b0, b1);
        if (i < live) w[i] = ya;
        if (i + 1 < live) w[i + 1] = yb;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The 8 split pairs of two vectors (first and second half of the rotated
// columns), one by one: packed, the registers cost more than the issue gains
// (18,900 rows of 12 heads of 128: 23.9 us, packed 24.9).
__device__ __forceinline__ void turn_halves(uint4& a, uint4& b, const float (&c)[8], const float (&s)[8]) {
    uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float p0 = lo_f(u[i]), p1 = hi_f(u[i]), q0 = lo_f(v[i]), q1 = hi_f(v[i]);
        u[i] = ptx::pack_bf16(fmaf(p0, c[2 * i], -(q0 * s[2 * i])), fmaf(p1, c[2 * i + 1], -(q1 * s[2 * i + 1])));
        v[i] = ptx::pack_bf16(fmaf(p0, s[2 * i], q0 * c[2 * i]), fmaf(p1, s[2 * i + 1], q1 * c[2 * i + 1]));
    }
    a = make_uint4(u[0], u[1], u[2], u[3]);
    b = make_uint4(v[0], v[1], v[2], v[3]);
}

// kHalves: a unit of a rotated tensor is the vector pair of 8 split pairs
// (units past the rotated columns are single vectors).  kFixed: the units of
// a head divide 32, so a lane's slots are the same in every head.
template <bool kHalves, bool kFixed>
__global__ void __launch_bounds__(kWarps * 32)
rope_rows_kernel(const __grid_constant__ Args a) {
    // units in flight per lane: more cost occupancy, fewer leave gaps (Q, K and V
    // of 11,466 rows of 12 heads of 128: 36.5 us with 4, 35.1 with 6, 41.0 with 8)
    constexpr int kUnroll = kHalves ? 4 : 6;
    const int lane = threadIdx.x & 31;
    const unsigned item = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const unsigned rj = item / (unsigned)a.parts;
    const int part = (int)(item - rj * (unsigned)a.parts);
    const int r = (int)(rj / (unsigned)a.n_jobs);
    // Launched before the kernel in front has ended (Q, K and V of 11,466 rows,
    // call after call: 36.3 us each, 37.6 without): nothing in global memory is
    // touched before the wait.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (r >= a.n_rows) return;
    const Job& jb = a.job[rj - (unsigned)r * (unsigned)a.n_jobs];
    // the row's id is asked for first: what follows from it arrives with the row
    const int id = a.at.ids ? __ldg(a.at.ids + r) : r;
    const int id_before = a.at.ascending && r > 0 ? __ldg(a.at.ids + r - 1) : -1;

    constexpr int kN = kHalves ? 8 : 4;                    // slots of a unit
    const bool rot = jb.rotate != 0;
    const bool split = kHalves && rot;
    const int half_vec = a.tab.slots / 8;                  // vectors of one half (halves pairing)
    const int units = split ? a.d_vec - half_vec : a.d_vec;   // units of a head
    const int total = units * jb.heads;
    const int share = ((total + a.parts - 1) / a.parts + 31) / 32 * 32;
    const int begin = part * share, end = min(total, begin + share);
    if (begin >= end) return;

    const uint4* src = jb.src + (long long)r * jb.src_ld;
    // Unit e is unit e % units of head e / units; the second vector of a split
    // pair lies half_vec further on.  kFixed: 32 units on, the same unit of a
    // later head, so both addresses go up by constants (the division by a
    // runtime `units` for every unit kept 71% of the issue slots busy).
    const int shift = kFixed ? __ffs(units) - 1 : 0;
    auto head_of = [&](int e) { return kFixed ? e >> shift : e / units; };
    auto col_of = [&](int u) { return split && u >= half_vec ? u + half_vec : u; };
    const int my_unit = kFixed ? lane & (units - 1) : 0, my_col = col_of(my_unit);
    const int src_step = kFixed ? (32 >> shift) * a.d_vec : 0;
    uint4 x[kUnroll], y[kHalves ? kUnroll : 1];
    auto load = [&](int e0) {
        const uint4* at = kFixed ? src + head_of(e0) * a.d_vec + my_col : src;
#pragma unroll
        for (int q = 0; q < kUnroll; ++q) {
            const int e = e0 + 32 * q;
            if (e < end) {
                const int u = kFixed ? my_unit : e % units;
                const uint4* s = kFixed ? at + q * src_step : src + head_of(e) * a.d_vec + col_of(u);
                x[q] = *s;
                if (kHalves && split && u < half_vec) y[q] = s[half_vec];
            }
        }
    };
    int e0 = begin + lane;
    load(e0);                                              // in flight while the row is resolved

    int p[3] = {0, 0, 0};
    long long base = 0;
    if (!resolve(a, r, id, id_before, p, base)) return;
    uint4* dst = jb.dst + (jb.cached ? base : (long long)r * jb.dst_ld);
    float c[kN], s[kN];
    if (kFixed && rot) load_cs<kN>(a.tab, p, my_unit * kN, c, s);

    const long long dst_step = kFixed ? (32 >> shift) * jb.dst_head : 0;
    for (;;) {
        uint4* at = kFixed ? dst + head_of(e0) * jb.dst_head + my_col : dst;
#pragma unroll
        for (int q = 0; q < kUnroll; ++q) {
            const int e = e0 + 32 * q;
            if (e >= end) continue;
            const int u = kFixed ? my_unit : e % units;
            uint4* d = kFixed ? at + q * dst_step : dst + head_of(e) * jb.dst_head + col_of(u);
            if (rot) {
                if (!kFixed) load_cs<kN>(a.tab, p, u * kN, c, s);
                if constexpr (kHalves) {
                    if (u < half_vec) {
                        turn_halves(x[q], y[q], c, s);
                        d[half_vec] = y[q];
                    }
                } else {
                    x[q] = turn_pairs(x[q], c, s, a.tab.slots - u * 4);
                }
            }
            *d = x[q];
        }
        e0 += 32 * kUnroll;
        if (e0 >= end) break;
        load(e0);
    }
}

// One thread per table entry: the angle in fp64, its cos and sin rounded once.
__global__ void __launch_bounds__(256)
rope_table_kernel(const __grid_constant__ Tab t, double theta, int shared_freq, float2* out, int n) {
    const int e = blockIdx.x * 256 + threadIdx.x;
    if (e >= n) return;
    int x = 0, first = 0, i = e, slot0 = 0;
    while (x < 2 && i >= t.np[x] * t.ns[x]) {
        first += t.np[x] * t.ns[x];
        slot0 += t.ns[x];
        i = e - first;
        ++x;
    }
    const int pos = i / t.ns[x], slot = i % t.ns[x];
    const double f = shared_freq ? (double)(slot0 + slot) / t.slots : (double)slot / t.ns[x];
    double s, c;
    sincos(pos * pow(theta, -f), &s, &c);
    out[e] = make_float2((float)c, (float)s);
}

Tab make_tab(const jano_rope_cfg& c, const float* table) {
    Tab t{};
    t.cs = reinterpret_cast<const float2*>(table);
    for (int x = 0; x < 3; ++x) {
        t.ns[x] = c.axes[x] / 2;
        t.np[x] = c.n_pos[x];
        t.slots += t.ns[x];
    }
    return t;
}

bool power_of_two_to_32(int u) { return u >= 1 && u <= 32 && 32 % u == 0; }

cudaError_t launch_rows(Args& a, bool halves, cudaStream_t st) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // whole rows per warp while they give each SM 32 warps; fewer rows are cut
    // into parts of at least 32 units
    const int half_vec = halves ? a.tab.slots / 8 : 0;
    int most = 1;
    bool fixed = true;
    for (int j = 0; j < a.n_jobs; ++j) {
        const int units = halves && a.job[j].rotate ? a.d_vec - half_vec : a.d_vec;
        const int p = (units * a.job[j].heads + 31) / 32;
        most = p > most ? p : most;
        fixed = fixed && power_of_two_to_32(units);
    }
    const long long warps = (long long)a.n_rows * a.n_jobs;
    const long long want = ((long long)sms * 32 + warps - 1) / warps;
    a.parts = (int)(want < 1 ? 1 : (want > most ? most : want));
    const long long blocks = (warps * a.parts + kWarps - 1) / kWarps;
    if (warps * a.parts > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (halves)
        return fixed ? cudaLaunchKernelEx(&cfg, rope_rows_kernel<true, true>, a)
                     : cudaLaunchKernelEx(&cfg, rope_rows_kernel<true, false>, a);
    return fixed ? cudaLaunchKernelEx(&cfg, rope_rows_kernel<false, true>, a)
                 : cudaLaunchKernelEx(&cfg, rope_rows_kernel<false, false>, a);
}

Job make_job(const void* src, long long src_ld, void* dst, long long dst_ld, long long dst_head, int heads,
             bool rotate, bool cached) {
    Job j{};
    j.src = static_cast<const uint4*>(src);
    j.dst = static_cast<uint4*>(dst);
    j.src_ld = src_ld / 8;
    j.dst_ld = dst_ld / 8;
    j.dst_head = dst_head / 8;
    j.heads = heads;
    j.rotate = rotate;
    j.cached = cached;
    return j;
}

}  // namespace

cudaError_t launch_rope_table(const jano_rope_cfg& c, double theta, int shared_freq, float* table, cudaStream_t st) {
    const Tab t = make_tab(c, nullptr);
    const int n = t.np[0] * t.ns[0] + t.np[1] * t.ns[1] + t.np[2] * t.ns[2];
    rope_table_kernel<<<(n + 255) / 256, 256, 0, st>>>(t, theta, shared_freq, reinterpret_cast<float2*>(table), n);
    return cudaGetLastError();
}

cudaError_t launch_axis_rope(const void* x, long long x_ld, const int32_t* ids, const int32_t* coords, int n_rows,
                             int heads, int d, const jano_rope_cfg& c, const float* table, void* out,
                             long long out_ld, int* err, cudaStream_t st) {
    Args a{};
    a.job[0] = make_job(x, x_ld, out, out_ld, d, heads, true, false);
    a.n_jobs = 1;
    a.n_rows = n_rows;
    a.d_vec = d / 8;
    a.tab = make_tab(c, table);
    a.at.ids = ids;
    a.at.coords = coords;
    a.at.grid_h = c.grid_h;
    a.at.grid_w = c.grid_w;
    a.err = err;
    return launch_rows(a, c.halves != 0, st);
}

cudaError_t launch_rope_cache(const RopeCacheCall& r, int* err, cudaStream_t st) {
    Args a{};
    const bool rotate = r.cfg != nullptr;
    if (r.q) a.job[a.n_jobs++] = make_job(r.q, r.q_ld, r.q_out, r.q_out_ld, r.d, r.heads, rotate, false);
    a.job[a.n_jobs++] = make_job(r.k, r.k_ld, r.k_cache, 0, r.head_stride, r.kv_heads, rotate, true);
    a.job[a.n_jobs++] = make_job(r.v, r.v_ld, r.v_cache, 0, r.head_stride, r.kv_heads, false, true);
    a.n_rows = r.n_rows;
    a.d_vec = r.d / 8;
    if (rotate) {
        a.tab = make_tab(*r.cfg, r.table);
        a.at.grid_h = r.cfg->grid_h;
        a.at.grid_w = r.cfg->grid_w;
    }
    a.at.ids = r.ids;
    a.at.coords = r.coords;
    a.at.grids = r.grids;
    a.at.ascending = 1;
    a.at.n_tokens = r.n_tokens;
    if (r.seqs) {
        a.at.table = r.seqs->page_table;
        a.at.lens = r.seqs->seq_lens;
        a.at.cu = r.seqs->cu_rows;
        a.at.n_seqs = r.seqs->n_seqs;
        a.at.max_pages = r.seqs->max_pages;
        a.at.n_pages = r.n_pages;
        while ((1 << a.at.page_shift) < r.page_size) ++a.at.page_shift;
    }
    a.at.page_stride = r.page_stride / 8;
    a.at.token_stride = r.token_stride / 8;
    a.at.head_stride = r.head_stride / 8;
    a.err = err;
    return launch_rows(a, rotate && r.cfg->halves, st);
}

}  // namespace jano
