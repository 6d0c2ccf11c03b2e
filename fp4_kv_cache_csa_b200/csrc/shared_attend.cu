// shared_attend.cu -- hca_shared_attend: dense attention of many queries over the
// compressed blocks of one cache slot (a prompt that many continuations share, a
// prefill chunk), joined with each query's own part.
//
// Per query and head: u_j = softmax_scale <q, e_j> over the visible blocks j,
// lse = ln sum_j exp(u_j), out = sum_j exp(u_j - lse) e_j; a second part with result
// (join_out, join_lse) over other entries joins by its log-sum-exp:
// L = ln(exp(lse) + exp(join_lse)), out = exp(lse - L) out + exp(join_lse - L) join_out.
//
// One tile product serves 64 columns, a column being one (query, head) of the slot: all
// 64 heads of a query, or as many whole queries as fit (H = 16: four). A tile of
// 128 blocks is so dequantized once per 64 columns, and no column is wasted on heads
// that a model does not have. Group = up to 64 columns; the flat list of all groups'
// tiles is cut into one range per CTA by cost, and groups that several CTAs share
// leave unnormalised partials for shared_merge_kernel.
//
// The products are transposed, as in attend.cu, because O of 64 columns x 512
// channels fills half of an SM's tensor memory in float32: S^T = E' Q'^T (M = 128
// blocks, N = 64 columns), O^T += E'^T P' (M = 128 channels, N = 64, K = 128 blocks).
// Operands are fp16: E'_j = e_j 2^-R_j and q' = q 2^-sQ are exact (R_j: the row's
// largest E8M0 exponent, 7 with E4M3 scales; sQ puts each column's max |q| into
// [2^14, 2^15)); P' = 2^(u log2 e + (R_j - B) - rho) <= 2^8, with B a common exponent, is
// rounded to fp16's 11 bits, which leaves about 1e-4 of the output's norm, an order
// below the bf16 rounding of the output. Row sums, references and accumulators are float32.
//
// Warp roles (13 warps, one CTA per SM): four dequantize (they also bring the
// group's queries in), eight do the softmax and the outputs, one thread issues the
// MMAs (a fourteenth warp or more would cut the registers of a thread from 128 to 96,
// and the softmax spills). What bounds it at D = 512: M = 128, N = 64 MMAs read 6 KB of operands from
// shared memory per 128 x 64 x 16 products, so shared memory (128 B/cycle) holds them to
// 0.63 of the tensor rate; the 128 KB tile of 128 blocks leaves no room for a second one,
// so a tile's parts (128 channels each) are replaced as its O^T products release
// them, and the tensor core waits while the softmax of a tile runs. At D = 128 three
// tiles fit and the softmax is the bound.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "tc_util.cuh"

namespace csa {

namespace {

constexpr int kTile = 128;  // blocks of a tile
constexpr int kCols = 64;   // columns of a group
constexpr int kSoftmaxWarps = 8, kDequantWarps = 4;
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kThreads = 32 * (kSoftmaxWarps + kDequantWarps + 1);
constexpr int kMmaWarp = kSoftmaxWarps + kDequantWarps;
// Row exponents count from B, the largest of the group's first tile in the CTA (127, that is 1, when
// its rows are all zero), and a row's is at least B - 40: what that flushes to zero lies below
// 2^-64 of the first tile's scale, and no sum leaves float32's range over all-zero rows (scale byte 0)
constexpr int kExponentSpan = 40;
constexpr float kNoRho = -1e30f;  // reference of a column that has not met an entry
// cost units by which the tile list is shared out: a tile, and the start of a group (its queries, its output)
constexpr long long kTileUnits = 100, kStartUnits = 150;
constexpr int kScaleE8M0x32 = 0, kScaleE4M3x16 = 1;

template <int D>
struct Cfg {
    static constexpr int PARTS = D / 128;                // parts of a tile: 128 channels each
    static constexpr int NBUF = D == 512 ? 1 : 3;        // tiles in shared memory
    static constexpr int NP = NBUF == 1 ? 1 : 2;         // P' buffers
    static constexpr int E_BYTES = kTile * D * 2;
    static constexpr int Q_BYTES = kCols * D * 2;
    static constexpr int P_BYTES = kTile * kCols * 2;
    static constexpr int SLICE = kTile * 128;            // 64 channels of a tile
    static constexpr int QSLICE = kCols * 128;           // 64 channels of the queries
    static constexpr int TMEM_O = 2 * kCols;             // S^T twice, then O^T
    static constexpr int TMEM_COLS = TMEM_O + PARTS * kCols <= 256 ? 256 : 512;
    static constexpr int MISC = 6144;
    static constexpr int SMEM = 1024 + NBUF * E_BYTES + Q_BYTES + NP * P_BYTES + MISC;
};

// A group of columns: queries q0 .. q0 + nq - 1 of slot b, its tiles [t0, t1) of the flat list.
struct Group {
    int b, q0, nq, n_max;  // n_max / n_min: most and fewest visible blocks of its queries
    int n_min, pad0, pad1, pad2;
    long long t0, t1;
};

struct SharedArgs {
    const uint8_t *fp4, *scale;
    const __nv_bfloat16 *q;
    const int32_t *q_offsets, *q_pos, *n_blocks;
    const float *join_out, *join_lse;
    __nv_bfloat16 *out;
    float *lse;
    int32_t *status;
    Group *groups;             // [groups_max]
    long long *gunits;         // [groups_max + 1] prefix of cost units
    int *gbase;                // [batch + 1] first group of each slot
    long long *cta_t;          // [G + 1] first tile of each CTA's range
    int *cta_g;                // [G] first group
    int *n_groups;
    float *part_o, *part_rho, *part_l;
    int batch, cap, m, Nq, H, per_group, G, groups_max;
    float scale_log2;
};

__device__ __forceinline__ int visible_of(const SharedArgs &a, int b, int i) {
    const int n = min(max(a.n_blocks[b], 0), a.cap);
    return a.q_pos ? min(visible_blocks(a.q_pos[i], a.m, n), n) : n;
}
__device__ __forceinline__ int query_bound(const SharedArgs &a, int b) { return min(max(a.q_offsets[b], 0), a.Nq); }

// ---------------------------------------------------------------- schedule
// One thread block: groups of every slot, their tiles, and the CTAs' ranges. A group
// without a visible block keeps one (wholly masked) tile, so that its output is written
// like any other.
__global__ void __launch_bounds__(1024) shared_schedule_kernel(SharedArgs a) {
    __shared__ long long tmp[32];
    __shared__ long long round_total;
    grid_dep_launch();
    long long carry = 0;
    for (int base = 0; base < a.batch; base += blockDim.x) {
        const int b = base + threadIdx.x;
        long long g = 0;
        if (b < a.batch) g = (max(query_bound(a, b + 1) - query_bound(a, b), 0) + a.per_group - 1) / a.per_group;
        const long long incl = block_inclusive_scan<long long>(g, tmp);
        if (b < a.batch) a.gbase[b + 1] = (int)min(carry + incl, (long long)a.groups_max);
        if (threadIdx.x == blockDim.x - 1) round_total = incl;
        __syncthreads();
        carry += round_total;
        __syncthreads();
    }
    if (threadIdx.x == 0) a.gbase[0] = 0;
    __threadfence_block();
    __syncthreads();
    const int NG = (int)min(carry, (long long)a.groups_max);  // groups_max only cuts offsets that are not ascending
    long long tcarry = 0, ucarry = 0;
    for (int base = 0; base < NG; base += blockDim.x) {
        const int g = base + threadIdx.x;
        long long tiles = 0, units = 0;
        Group r = {};
        if (g < NG) {
            int lo = 0, hi = a.batch - 1;  // the slot with gbase[b] <= g < gbase[b + 1]
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (a.gbase[mid + 1] <= g) lo = mid + 1; else hi = mid;
            }
            r.b = lo;
            r.q0 = query_bound(a, lo) + (g - a.gbase[lo]) * a.per_group;
            r.nq = min(a.per_group, query_bound(a, lo + 1) - r.q0);
            r.n_max = 0;
            r.n_min = 0x7fffffff;
            for (int k = 0; k < r.nq; ++k) {
                const int n = visible_of(a, lo, r.q0 + k);
                r.n_max = max(r.n_max, n);
                r.n_min = min(r.n_min, n);
            }
            tiles = max(1, (r.n_max + kTile - 1) / kTile);
            units = kStartUnits + kTileUnits * tiles;
        }
        const long long tin = block_inclusive_scan<long long>(tiles, tmp);
        if (g < NG) {
            r.t0 = tcarry + tin - tiles;
            r.t1 = tcarry + tin;
            a.groups[g] = r;
        }
        if (threadIdx.x == blockDim.x - 1) round_total = tin;
        __syncthreads();
        tcarry += round_total;
        __syncthreads();
        const long long uin = block_inclusive_scan<long long>(units, tmp);
        if (g < NG) a.gunits[g + 1] = ucarry + uin;
        if (threadIdx.x == blockDim.x - 1) round_total = uin;
        __syncthreads();
        ucarry += round_total;
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        a.gunits[0] = 0;
        *a.n_groups = NG;
    }
    __threadfence_block();
    __syncthreads();
    // CTA c begins at the tile boundary nearest to its share of the units
    for (int c = threadIdx.x; c <= a.G; c += blockDim.x) {
        long long t = tcarry;
        int first = max(NG - 1, 0);
        if (c < a.G && NG > 0) {
            const long long ub = ucarry * c / a.G;
            int lo = 0, hi = NG - 1;  // last group with gunits[g] <= ub
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (a.gunits[mid] <= ub) lo = mid; else hi = mid - 1;
            }
            const Group r = a.groups[lo];
            const long long x = ub - a.gunits[lo] - kStartUnits;
            const long long k = x > 0 ? min((x + kTileUnits / 2) / kTileUnits, r.t1 - r.t0) : 0;
            t = r.t0 + k;
            first = t == r.t1 && lo + 1 < NG ? lo + 1 : lo;
        }
        a.cta_t[c] = t;
        if (c < a.G) a.cta_g[c] = first;
    }
}

// ---------------------------------------------------------------- operands
// The channel that lane position `pos` of a d-tile holds (dequantization may permute channels within
// a tile as long as queries and outputs follow).
__device__ __forceinline__ int channel_of(int pos) { return pos; }

// One row's codes (128 channels of each part) and its scales, held by one thread.
template <int D, int SF>
struct Row {
    static constexpr int SW = SF == 0 ? Cfg<D>::PARTS : 2 * Cfg<D>::PARTS;  // 32-bit words of scales
    uint4 code[Cfg<D>::PARTS][4];
    uint32_t sc[SW];
    bool valid;
};

template <int D, int SF>
__device__ __forceinline__ void load_scales(const SharedArgs &a, size_t row, Row<D, SF> &r) {
    constexpr int SW = Row<D, SF>::SW;
    const uint8_t *src = a.scale + row * (4 * SW);
    if constexpr (SW >= 4) {
#pragma unroll
        for (int k = 0; k < SW; k += 4) {
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(src) + k / 4);
            r.sc[k] = u.x;
            r.sc[k + 1] = u.y;
            r.sc[k + 2] = u.z;
            r.sc[k + 3] = u.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < SW; ++k) r.sc[k] = __ldg(reinterpret_cast<const uint32_t *>(src) + k);
    }
}

template <int D, int SF>
__device__ __forceinline__ void load_codes(const SharedArgs &a, size_t row, int p, Row<D, SF> &r) {
    const uint4 *src = reinterpret_cast<const uint4 *>(a.fp4 + row * (D / 2) + p * 64);
#pragma unroll
    for (int k = 0; k < 4; ++k) r.code[p][k] = __ldg(src + k);
}

// The largest scale exponent byte of the row (E8M0).
template <int N>
__device__ __forceinline__ int row_exponent(const uint32_t (&sc)[N]) {
    uint32_t m = sc[0];
#pragma unroll
    for (int k = 1; k < N; ++k) m = __vmaxu4(m, sc[k]);
    m = __vmaxu4(m, m >> 16);
    m = __vmaxu4(m, m >> 8);
    return (int)(m & 0xFF);
}

// One part of the row (128 channels, two slices of the buffer) into E', fp16, in the
// 128-byte-swizzled layout of the MMA.
template <int D, int SF>
__device__ __forceinline__ void dequant(const uint4 (&code)[4], const uint32_t (&sc)[Row<D, SF>::SW], int rmax, int p,
                                        int j, uint8_t *E) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {  // 32 channels: half a slice
        uint8_t *to = E + (2 * p + (v >> 1)) * Cfg<D>::SLICE + (j >> 3) * 1024 + (j & 7) * 128;
        __half2 s2[2];
        if constexpr (SF == kScaleE8M0x32) {
            const int k = (int)((sc[p] >> (8 * v)) & 0xFF) - rmax;  // <= 0
            // 2^k in fp16: normal for k >= -14, subnormal down to -24, else 0
            const uint16_t hb = k >= -14 ? (uint16_t)((k + 15) << 10) : k >= -24 ? (uint16_t)(1u << (k + 24)) : 0;
            s2[0] = s2[1] = __halves2half2(__ushort_as_half(hb), __ushort_as_half(hb));
        } else {
            // E' = e 2^-7
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t byte = (sc[2 * p + (v >> 1)] >> (8 * (2 * (v & 1) + h))) & 0xFF;
                const __half_raw hr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3);
                const __half s = __hmul(__half(hr), __ushort_as_half((uint16_t)((15 - 7) << 10)));
                s2[h] = __halves2half2(s, s);
            }
        }
        const uint32_t w[4] = {code[v].x, code[v].y, code[v].z, code[v].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t o[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                __half2_raw hr = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((w[k] >> (8 * b)) & 0xFF), __NV_E2M1);
                const __half2 h = __hmul2(*reinterpret_cast<__half2 *>(&hr), s2[k >> 1]);
                o[b] = *reinterpret_cast<const uint32_t *>(&h);
            }
            *reinterpret_cast<uint4 *>(to + (((4 * (v & 1) + k) ^ (j & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// ---------------------------------------------------------------- main kernel
// B + 127 from what the dequantizing warps found (E8M0).
__device__ __forceinline__ int base_of(const int (&b)[4]) {
    const int m = max(max(b[0], b[1]), max(b[2], b[3]));
    return m > 0 ? m : 127;
}

// lse of a column, and the factor of its accumulator, from its reference and row sum; joined with
// another part's lse (jf: that part's factor).
__device__ __forceinline__ void finish(float rho, float l, bool join, float other, float &lse, float &f, float &jf) {
    const bool any = l > 0.f || l != l;  // (a NaN goes on)
    lse = any ? (rho + log2f(l)) * 0.69314718055994531f : -INFINITY;
    f = any ? 1.f / l : 0.f;
    jf = 0.f;
    if (join) {
        const float top = fmaxf(lse, other);
        if (top != -INFINITY) {
            const float x = expf(lse - top), y = expf(other - top);
            f *= x / (x + y);
            jf = y / (x + y);
            lse = top + logf(x + y);
        }
    }
}

// Where a role stands in the CTA's range.
struct Cursor {
    int g, seg;           // group, and its number within the CTA
    long long t, end;     // tile, end of the group's tiles within the range
    bool first;           // first tile of the group within the CTA
};

// Shared state behind the operand buffers.
struct Misc {
    uint64_t e_full[3][4], e_free[3][4], s_full[2], s_free[2], p_full[2], pv_done[2], q_full, q_free, o_free[2], r_full, drain;
    uint32_t tmem;
    int abort;
    alignas(16) float rho[kCols], alpha[kCols], fac[kCols], jfac[kCols];
    float wred[4][kCols];
    float colmul[2][kCols];  // scale_log2 * 2^(sQ + B) of each column, by segment parity
    int nvis[2][kCols];
    float rexp[3][kTile];    // R_j - B
    int base[2][4];          // largest exponent byte of each dequantizing warp's rows, by segment parity
};
static_assert(sizeof(Misc) <= 6144, "Misc exceeds its space");

template <int D, int SF>
__global__ void __launch_bounds__(kThreads, 1) shared_attend_kernel(const __grid_constant__ SharedArgs a) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *E = smem;
    uint8_t *Q = E + C::NBUF * C::E_BYTES;
    uint8_t *P = Q + C::Q_BYTES;
    Misc *ms = reinterpret_cast<Misc *>(P + C::NP * C::P_BYTES);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int b = 0; b < C::NBUF; ++b)
            for (int p = 0; p < C::PARTS; ++p) {
                mbar_init(smem_u32(&ms->e_full[b][p]), kDequantWarps);
                mbar_init(smem_u32(&ms->e_free[b][p]), 1);
            }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&ms->s_full[b]), 1);
            mbar_init(smem_u32(&ms->s_free[b]), kSoftmaxWarps);
            mbar_init(smem_u32(&ms->p_full[b]), kSoftmaxWarps);
            mbar_init(smem_u32(&ms->pv_done[b]), 1);
            mbar_init(smem_u32(&ms->o_free[b]), kSoftmaxWarps);
        }
        mbar_init(smem_u32(&ms->q_full), kDequantWarps);
        mbar_init(smem_u32(&ms->r_full), kDequantWarps);
        mbar_init(smem_u32(&ms->q_free), 1);
        mbar_init(smem_u32(&ms->drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        ms->abort = 0;
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ms->tmem)),
                     "r"(C::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms->tmem;
    const volatile int *abort = &ms->abort;
    grid_dep_wait();
    grid_dep_launch();
    const long long t_begin = a.cta_t[blockIdx.x], t_end = a.cta_t[blockIdx.x + 1];

    auto start = [&]() {
        Cursor c;
        c.g = a.cta_g[blockIdx.x];
        c.seg = 0;
        c.t = t_begin;
        c.end = min(t_end, a.groups[c.g].t1);
        c.first = true;
        return c;
    };
    // the next tile; the caller checks c.t < t_end
    auto step = [&](Cursor &c) {
        ++c.t;
        c.first = false;
        if (c.t >= c.end && c.t < t_end) {
            ++c.g;
            ++c.seg;
            c.end = min(t_end, a.groups[c.g].t1);
            c.first = true;
        }
    };

    if (t_begin >= t_end) {
        // nothing to do: fall through to the common end
    } else if (warp < kSoftmaxWarps) {
        // ================================================================ softmax and output
        const int j = tid & (kTile - 1), hf = tid >> 7;
        const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t s_addr = tmem + lane_off + 32 * hf;
        const uint32_t o_addr = tmem + lane_off + C::TMEM_O + 32 * hf;
        float lsum[32];
        int n = 0;  // tiles done by this CTA
        Cursor c = start();
        while (c.t < t_end) {
            const Group gr = a.groups[c.g];
            const int seg = c.seg, mp = seg & 1;
            const long long seg_begin = c.t;
            bool gave_up = false;
#pragma unroll
            for (int k = 0; k < 32; ++k) lsum[k] = 0.f;
            while (true) {
                const bool first = c.first;
                const int buf = n % C::NBUF, sb = n & 1, use = n / C::NBUF;
                bool ok = mbar_wait_ab<false>(smem_u32(&ms->e_full[buf][0]), use & 1, abort);
                ok = ok && mbar_wait_ab<false>(smem_u32(&ms->s_full[sb]), (n >> 1) & 1, abort);
                if (n >= C::NP)  // P' is free: the O^T product of tile n - NP is done
                    ok = ok && mbar_wait_ab<false>(smem_u32(&ms->pv_done[(n - C::NP) & 1]), ((n - C::NP) >> 1) & 1, abort);
                tc_fence_after();
                const float R = ms->rexp[buf][j];
                const float rmul = exp2f(R);  // R: the row's exponent from B on
                const int entry = (int)(c.t - gr.t0) * kTile + j;
                const bool masked = entry - j + kTile > gr.n_min;
                float u[32];
                auto logits = [&]() {  // u of this thread's 32 columns, from S^T; returns the largest u - rho
                    float over = -INFINITY;
                    tmem_ld32(s_addr + kCols * sb, u);
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        const float4 cm = *reinterpret_cast<const float4 *>(&ms->colmul[mp][32 * hf + k]);
                        const float4 rh = *reinterpret_cast<const float4 *>(&ms->rho[32 * hf + k]);
                        u[k] = fmaf(u[k], cm.x * rmul, R);
                        u[k + 1] = fmaf(u[k + 1], cm.y * rmul, R);
                        u[k + 2] = fmaf(u[k + 2], cm.z * rmul, R);
                        u[k + 3] = fmaf(u[k + 3], cm.w * rmul, R);
                        if (masked) {
                            const int4 nv = *reinterpret_cast<const int4 *>(&ms->nvis[mp][32 * hf + k]);
                            if (entry >= nv.x) u[k] = -INFINITY;
                            if (entry >= nv.y) u[k + 1] = -INFINITY;
                            if (entry >= nv.z) u[k + 2] = -INFINITY;
                            if (entry >= nv.w) u[k + 3] = -INFINITY;
                        }
                        over = fmaxf(over, fmaxf(fmaxf(u[k] - rh.x, u[k + 1] - rh.y), fmaxf(u[k + 2] - rh.z, u[k + 3] - rh.w)));
                    }
                    return over;
                };
                const float over = logits();
                // references: set by the group's first tile, raised (with O^T and the sums) when a
                // logit exceeds one by more than 8; a wait that ran out comes this way too
                if (bar_or_n<kSoftmaxThreads>(first || over > 8.f || !ok)) {
                    if (!first && n > 0)
                        ok = ok && mbar_wait_ab<false>(smem_u32(&ms->pv_done[(n - 1) & 1]), ((n - 1) >> 1) & 1, abort);
                    transpose_reduce32<true>(u);  // lane L: column 32 hf + L over this warp's entries
                    ms->wred[warp & 3][32 * hf + lane] = u[0];
                    if (bar_or_n<kSoftmaxThreads>(!ok)) {
                        ms->abort = 1;
                        gave_up = true;
                        break;
                    }
                    if (tid < kCols) {
                        const float M = fmaxf(fmaxf(ms->wred[0][tid], ms->wred[1][tid]),
                                              fmaxf(ms->wred[2][tid], ms->wred[3][tid]));
                        float al = 1.f;
                        if (first) {
                            ms->rho[tid] = fmaxf(M, kNoRho);
                        } else if (M > ms->rho[tid] + 8.f) {
                            al = exp2f(ms->rho[tid] - M);
                            ms->rho[tid] = M;
                        }
                        ms->alpha[tid] = al;
                    }
                    bar_sync_n<kSoftmaxThreads>();
                    if (!first) {
                        tc_fence_after();
#pragma unroll 1
                        for (int dt = 0; dt < C::PARTS; ++dt) {
                            float o[32];
                            tmem_ld32(o_addr + kCols * dt, o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] *= ms->alpha[32 * hf + k];
                            tmem_st32(o_addr + kCols * dt, o);
                        }
#pragma unroll
                        for (int k = 0; k < 32; ++k) lsum[k] *= ms->alpha[32 * hf + k];
                    }
                    logits();  // again: the reduction used them up (rare, and cheaper than registers for both)
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ms->s_free[sb]));
                // P' = 2^(u - rho), fp16, and the row sums (without 2^R_j, which P' carries for E')
                const float rinv = exp2f(-R);
                uint8_t *Pn = P + (n % C::NP) * C::P_BYTES + (j >> 3) * 1024 + (j & 7) * 128;
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) {
                    uint32_t pk[4];
#pragma unroll
                    for (int q2 = 0; q2 < 4; ++q2) {
                        const int k = 8 * cc + 2 * q2;
                        const float2 rh = *reinterpret_cast<const float2 *>(&ms->rho[32 * hf + k]);
                        const float p0 = exp2f(u[k] - rh.x), p1 = exp2f(u[k + 1] - rh.y);
                        const __half2 hh = __floats2half2_rn(p0, p1);
                        pk[q2] = *reinterpret_cast<const uint32_t *>(&hh);
                        lsum[k] = fmaf(p0, rinv, lsum[k]);
                        lsum[k + 1] = fmaf(p1, rinv, lsum[k + 1]);
                    }
                    *reinterpret_cast<uint4 *>(Pn + (((4 * hf + cc) ^ (j & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ms->p_full[n % C::NP]));
                ++n;
                step(c);
                if (c.first || c.t >= t_end) break;  // the group's last tile here
            }
            if (gave_up) break;
            // ---------------- the group's output, or its partial
            transpose_reduce32<false>(lsum);
            ms->wred[warp & 3][32 * hf + lane] = lsum[0];
            const bool ok = mbar_wait_ab<false>(smem_u32(&ms->pv_done[(n - 1) & 1]), ((n - 1) >> 1) & 1, abort);
            if (bar_or_n<kSoftmaxThreads>(!ok)) {
                ms->abort = 1;
                break;
            }
            const bool whole = seg_begin == gr.t0 && min(t_end, gr.t1) == gr.t1;
            const int cols = gr.nq * a.H;
            const size_t row0 = (size_t)gr.q0 * a.H;
            // O^T holds E' = e 2^-(R - B) times P' over 2^B
            const float unit = SF == kScaleE8M0x32 ? exp2f((float)(base_of(ms->base[mp]) - 127)) : exp2f(7.f);
            const int slot = 2 * blockIdx.x + (seg_begin == t_begin ? 0 : 1);
            if (tid < kCols) {
                const float l = ms->wred[0][tid] + ms->wred[1][tid] + ms->wred[2][tid] + ms->wred[3][tid];
                const float rho = ms->rho[tid];
                if (!whole) {
                    a.part_rho[(size_t)slot * kCols + tid] = rho;
                    a.part_l[(size_t)slot * kCols + tid] = l;
                } else if (tid < cols) {
                    float lse, f, jf;
                    finish(rho, l, a.join_lse != nullptr, a.join_lse ? a.join_lse[row0 + tid] : 0.f, lse, f, jf);
                    ms->fac[tid] = f;
                    ms->jfac[tid] = jf;
                    if (a.lse) a.lse[row0 + tid] = lse;
                }
            }
            bar_sync_n<kSoftmaxThreads>();
            tc_fence_after();
#pragma unroll 1
            for (int dt = 0; dt < C::PARTS; ++dt) {
                float o[32];
                tmem_ld32(o_addr + kCols * dt, o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] *= unit;
                if (dt == C::PARTS - 1) {  // O^T is read: the next group's products may start
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&ms->o_free[seg & 1]));
                }
                const int ch = channel_of(128 * dt + 32 * (warp & 3) + lane);
                if (!whole) {
                    float *dst = a.part_o + ((size_t)slot * kCols + 32 * hf) * D + ch;
#pragma unroll
                    for (int k = 0; k < 32; ++k) dst[(size_t)k * D] = o[k];
                } else {
                    const float *jo = a.join_out + (row0 + 32 * hf) * D + ch;
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        float v[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int col = 32 * hf + k + e;
                            v[e] = ms->fac[col] > 0.f || ms->fac[col] != ms->fac[col] ? o[k + e] * ms->fac[col] : 0.f;
                            if (a.join_lse && col < cols && !(ms->jfac[col] == 0.f))
                                v[e] = fmaf(ms->jfac[col], jo[(size_t)(k + e) * D], v[e]);
                        }
                        // even lanes take column k, odd ones k + 1, with their neighbour's channel
                        const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? v[0] : v[1], 1);
                        const int col = 32 * hf + k + (lane & 1);
                        if (col < cols) {
                            const __nv_bfloat162 h = (lane & 1) ? __floats2bfloat162_rn(got, v[1]) : __floats2bfloat162_rn(v[0], got);
                            *reinterpret_cast<__nv_bfloat162 *>(a.out + (row0 + col) * D + (ch & ~1)) = h;
                        }
                    }
                }
            }
            bar_sync_n<kSoftmaxThreads>();  // rho, fac, wred belong to the next group from here on
        }
    } else if (warp < kMmaWarp) {
        // ================================================================ dequantization, queries
        const int j = tid - kSoftmaxThreads, dw = warp - kSoftmaxWarps;
        Row<D, SF> r;
        Cursor c = start();
        Group gr = a.groups[c.g];
        // the row this thread dequantizes in a tile of a group, or -1
        auto row_of = [&](const Group &g, long long t) -> long long {
            const int e = (int)(t - g.t0) * kTile + j;
            return e < g.n_max ? (long long)g.b * a.cap + e : -1;
        };
        long long row = row_of(gr, c.t);
        r.valid = row >= 0;
        if (r.valid) {
            load_scales<D, SF>(a, row, r);
#pragma unroll
            for (int p = 0; p < C::PARTS; ++p) load_codes<D, SF>(a, row, p, r);
        }
        int n = 0, base = 127 + 7;
        bool ok = true;
        while (c.t < t_end) {
            if (c.first) {
                // the queries of the group: column = row q0 * H + column of q; per column 2^-sQ
                if (c.seg >= 1) ok = mbar_wait_ab<false>(smem_u32(&ms->q_free), (c.seg - 1) & 1, abort);
                if (c.seg >= 2) ok = ok && mbar_wait_ab<false>(smem_u32(&ms->o_free[c.seg & 1]), ((c.seg - 2) >> 1) & 1, abort);
                if (!__all_sync(0xffffffffu, ok)) break;
                const int cols = gr.nq * a.H, mp = c.seg & 1;
                if constexpr (SF == kScaleE8M0x32) {  // B, from the rows of the group's first tile
                    const int mine = __reduce_max_sync(0xffffffffu, r.valid ? row_exponent(r.sc) : 0);
                    if (lane == 0) {
                        ms->base[mp][dw] = mine;
                        mbar_arrive(smem_u32(&ms->r_full));
                    }
                    ok = mbar_wait_ab<false>(smem_u32(&ms->r_full), c.seg & 1, abort);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    base = base_of(ms->base[mp]);
                }
                constexpr int LANES = D == 512 ? 32 : 16;      // lanes of a column
                constexpr int PER = 32 / LANES;                // columns of a warp at a time
                constexpr int CH = D / 8 / LANES;              // 16-byte chunks of a lane
                const int sub = lane / LANES, sl = lane % LANES;
#pragma unroll 1
                for (int k0 = 0; k0 < kCols / kDequantWarps; k0 += 4 * PER) {
                    uint4 v[4][CH];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int col = dw * (kCols / kDequantWarps) + k0 + x * PER + sub;
                        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + ((size_t)gr.q0 * a.H + col) * D);
#pragma unroll
                        for (int y = 0; y < CH; ++y)
                            v[x][y] = col < cols ? __ldg(src + sl + y * LANES) : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int col = dw * (kCols / kDequantWarps) + k0 + x * PER + sub;
                        // max |q| as the largest bit pattern (bf16 magnitudes order like integers)
                        uint32_t mx = 0;
#pragma unroll
                        for (int y = 0; y < CH; ++y) {
                            const uint32_t *w = reinterpret_cast<const uint32_t *>(&v[x][y]);
#pragma unroll
                            for (int z = 0; z < 4; ++z) mx = __vmaxu2(mx, w[z] & 0x7FFF7FFFu);
                        }
                        mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
                        for (int o = LANES / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        const int sq = mx > 0 ? max((int)(mx >> 7) - 127 - 14, -126) : 0;  // (2^126 is still a float32)
                        const float inv = ldexpf(1.0f, -sq);
#pragma unroll
                        for (int y = 0; y < CH; ++y) {
                            const int kc = sl + y * LANES;
                            const __nv_bfloat162 *h2 = reinterpret_cast<const __nv_bfloat162 *>(&v[x][y]);
                            uint32_t o[4];
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                const float2 f = __bfloat1622float2(h2[z]);
                                const __half2 hh = __floats2half2_rn(f.x * inv, f.y * inv);
                                o[z] = *reinterpret_cast<const uint32_t *>(&hh);
                            }
                            *reinterpret_cast<uint4 *>(Q + (kc >> 3) * C::QSLICE + (col >> 3) * 1024 + (col & 7) * 128 +
                                                       (((kc & 7) ^ (col & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                        if (sl == 0) {
                            ms->colmul[mp][col] = ldexpf(a.scale_log2, sq + base - 127);
                            ms->nvis[mp][col] = col < cols ? visible_of(a, gr.b, gr.q0 + col / a.H) : 0;
                        }
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ms->q_full));
            }
            // the tile after this one, whose rows are loaded as this one's registers empty
            Cursor nx = c;
            step(nx);
            const bool more = nx.t < t_end;
            Group gn = gr;
            if (more && nx.first) gn = a.groups[nx.g];
            const long long row_n = more ? row_of(gn, nx.t) : -1;

            const int buf = n % C::NBUF, use = n / C::NBUF;
            uint8_t *En = E + buf * C::E_BYTES;
            const bool valid = r.valid;
            const int rmax = SF == kScaleE8M0x32 && valid ? max(row_exponent(r.sc), base - kExponentSpan) : base;
#pragma unroll
            for (int p = 0; p < C::PARTS; ++p) {
                if (use >= 1) ok = mbar_wait_ab<false>(smem_u32(&ms->e_free[buf][p]), (use - 1) & 1, abort);
                if (!__all_sync(0xffffffffu, ok)) break;
                if (p == 0) ms->rexp[buf][j] = (float)(rmax - base);
                if (valid) {
                    dequant<D, SF>(r.code[p], r.sc, rmax, p, j, En);
                } else {
                    uint8_t *to = En + 2 * p * C::SLICE + (j >> 3) * 1024 + (j & 7) * 128;
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        *reinterpret_cast<uint4 *>(to + (k >> 3) * C::SLICE + ((k & 7) << 4)) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ms->e_full[buf][p]));
                if (row_n >= 0) load_codes<D, SF>(a, row_n, p, r);  // (this part's registers are free)
            }
            if (!__all_sync(0xffffffffu, ok)) break;
            r.valid = row_n >= 0;
            if (r.valid) load_scales<D, SF>(a, row_n, r);
            ++n;
            c = nx;
            gr = gn;
        }
        if (!ok) ms->abort = 1;
    } else if (lane == 0) {  // (the warp's other lanes wait at the common end)
        // ================================================================ MMA issue
        constexpr uint32_t IDESC_S = idesc_f16(kTile, kCols, false, false);
        constexpr uint32_t IDESC_O = idesc_f16(kTile, kCols, true, true);
        const uint32_t E_s = smem_u32(E), Q_s = smem_u32(Q), P_s = smem_u32(P);
        bool ok = true;
        // S^T of tile n
        auto score = [&](int n, const Cursor &c, bool last) {
            const int buf = n % C::NBUF, sb = n & 1, use = n / C::NBUF;
            if (c.first) ok = ok && mbar_wait_ab<false>(smem_u32(&ms->q_full), c.seg & 1, abort);
            if (n >= 2) ok = ok && mbar_wait_ab<false>(smem_u32(&ms->s_free[sb]), ((n >> 1) - 1) & 1, abort);
            for (int p = 0; p < C::PARTS; ++p) {
                ok = ok && mbar_wait_ab<false>(smem_u32(&ms->e_full[buf][p]), use & 1, abort);
                if (!ok) return;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {  // 16 channels each
                    const int sl = 2 * p + (kk >> 2);
                    const uint64_t da = desc_sw128(E_s + buf * C::E_BYTES + sl * C::SLICE + (kk & 3) * 32, 16, 1024);
                    const uint64_t db = desc_sw128(Q_s + sl * C::QSLICE + (kk & 3) * 32, 16, 1024);
                    mma_f16(tmem + kCols * sb, da, db, IDESC_S, p > 0 || kk > 0);
                }
            }
            mma_commit(smem_u32(&ms->s_full[sb]));
            if (last) mma_commit(smem_u32(&ms->q_free));
        };
        // O^T += of tile n
        auto value = [&](int n, const Cursor &c) {
            const int buf = n % C::NBUF;
            ok = ok && mbar_wait_ab<false>(smem_u32(&ms->p_full[n % C::NP]), (n / C::NP) & 1, abort);
            if (c.first && c.seg >= 1) ok = ok && mbar_wait_ab<false>(smem_u32(&ms->o_free[(c.seg - 1) & 1]), ((c.seg - 1) >> 1) & 1, abort);
            if (!ok) return;
            tc_fence_after();
#pragma unroll 1
            for (int p = 0; p < C::PARTS; ++p) {
#pragma unroll
                for (int kj = 0; kj < kTile / 16; ++kj) {  // 16 blocks each
                    const uint64_t da = desc_sw128(E_s + buf * C::E_BYTES + 2 * p * C::SLICE + kj * 2048, C::SLICE, 1024);
                    const uint64_t db = desc_sw128(P_s + (n % C::NP) * C::P_BYTES + kj * 2048, 8192, 1024);
                    mma_f16(tmem + C::TMEM_O + kCols * p, da, db, IDESC_O, !c.first || kj > 0);
                }
                mma_commit(smem_u32(&ms->e_free[buf][p]));
            }
            mma_commit(smem_u32(&ms->pv_done[n & 1]));
        };
        Cursor cs = start(), cv = cs;
        int ns = 0, nv = 0;
        while (cv.t < t_end && ok) {
            // with several tile buffers S^T runs one tile ahead of O^T
            while (ok && cs.t < t_end && ns < nv + (C::NBUF > 1 ? 2 : 1)) {
                Cursor nx = cs;
                step(nx);
                score(ns, cs, nx.first || nx.t >= t_end);
                cs = nx;
                ++ns;
            }
            if (!ok) break;
            value(nv, cv);
            step(cv);
            ++nv;
        }
        if (!ok) {
            ms->abort = 1;
            // nothing issued may still run when the CTA leaves
            mma_commit(smem_u32(&ms->drain));
            mbar_wait_for(smem_u32(&ms->drain), 0, kDrainCycles);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && ms->abort) flag(a.status, CSA_DEV_TIMEOUT);
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS) : "memory");
}

// ---------------------------------------------------------------- merge
// A group that several CTAs worked on: blockIdx.x + 1 is a CTA whose range begins inside the group, the
// first such CTA merges it. blockIdx.y: 8 columns, blockIdx.z: 128 channels.
constexpr int kMergeCols = 8, kMostParts = 256;

__global__ void __launch_bounds__(256) shared_merge_kernel(SharedArgs a, int D) {
    __shared__ int slots[kMostParts];
    __shared__ float wts[kMostParts * kMergeCols];
    __shared__ float s_join[kMergeCols];
    __shared__ int np_s;
    grid_dep_wait();
    const int c = blockIdx.x + 1, NG = *a.n_groups;
    const long long tb = a.cta_t[c];
    if (NG == 0) return;
    int lo = 0, hi = NG - 1;  // the group that holds tile tb - 1
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.groups[mid].t1 < tb) lo = mid + 1; else hi = mid;
    }
    const Group gr = a.groups[lo];
    if (tb <= gr.t0 || tb >= gr.t1) return;              // the boundary lies between two groups
    if (c > 1 && a.cta_t[c - 1] > gr.t0) return;         // an earlier CTA begins inside the group, too
    const int cols = gr.nq * a.H, c0 = blockIdx.y * kMergeCols;
    if (c0 >= cols) return;
    const int nc = min(kMergeCols, cols - c0);
    if (threadIdx.x < 32) {  // the CTAs with tiles of the group, in order (c - 1 holds its first ones)
        int np = 0;
        for (int base = c - 1; base < a.G; base += 32) {
            const int cc = base + (int)threadIdx.x;
            bool has = false;
            long long rb = 0;
            if (cc < a.G) {
                rb = a.cta_t[cc];
                has = rb < a.cta_t[cc + 1] && rb < gr.t1 && a.cta_t[cc + 1] > gr.t0;
            }
            const uint32_t mask = __ballot_sync(0xffffffffu, has);
            const int pos = np + __popc(mask & ((1u << threadIdx.x) - 1u));
            if (has && pos < kMostParts) slots[pos] = 2 * cc + (rb >= gr.t0 ? 0 : 1);
            np += __popc(mask);
            if (!__any_sync(0xffffffffu, cc < a.G && rb < gr.t1)) break;
        }
        if (threadIdx.x == 0) np_s = min(np, kMostParts);
    }
    __syncthreads();
    const int np = np_s;
    const int hh = threadIdx.x >> 5, lane = threadIdx.x & 31;  // one warp per column
    const size_t row0 = (size_t)gr.q0 * a.H + c0;
    if (hh < nc) {
        float top = -INFINITY;
        for (int p = lane; p < np; p += 32) top = fmaxf(top, a.part_rho[(size_t)slots[p] * kCols + c0 + hh]);
        top = warp_max(top);
        float l = 0.f;
        for (int p = lane; p < np; p += 32) {
            const size_t at = (size_t)slots[p] * kCols + c0 + hh;
            const float w = exp2f(a.part_rho[at] - top);
            wts[p * kMergeCols + hh] = w;
            l = fmaf(w, a.part_l[at], l);
        }
        l = warp_sum(l);
        float lse, f, jf;
        finish(top, l, a.join_lse != nullptr, a.join_lse ? a.join_lse[row0 + hh] : 0.f, lse, f, jf);
        __syncwarp();
        for (int p = lane; p < np; p += 32) wts[p * kMergeCols + hh] *= f;
        if (lane == 0) {
            s_join[hh] = jf;
            if (a.lse && blockIdx.z == 0) a.lse[row0 + hh] = lse;
        }
        __syncwarp();
        const int d4 = blockIdx.z * 32 + lane;  // four channels
        const float4 *src = reinterpret_cast<const float4 *>(a.part_o + (size_t)(c0 + hh) * D) + d4;
        const size_t stride = (size_t)kCols * D / 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p0 = 0; p0 < np; p0 += 8) {
            float4 o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                o[k] = p0 + k < np ? __ldcg(src + (size_t)slots[p0 + k] * stride) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float w = p0 + k < np ? wts[(p0 + k) * kMergeCols + hh] : 0.f;
                acc.x = fmaf(w, o[k].x, acc.x);
                acc.y = fmaf(w, o[k].y, acc.y);
                acc.z = fmaf(w, o[k].z, acc.z);
                acc.w = fmaf(w, o[k].w, acc.w);
            }
        }
        if (a.join_lse && !(s_join[hh] == 0.f)) {
            const float4 x = reinterpret_cast<const float4 *>(a.join_out + (row0 + hh) * D)[d4];
            acc.x = fmaf(s_join[hh], x.x, acc.x);
            acc.y = fmaf(s_join[hh], x.y, acc.y);
            acc.z = fmaf(s_join[hh], x.z, acc.z);
            acc.w = fmaf(s_join[hh], x.w, acc.w);
        }
        const __nv_bfloat162 h0 = __floats2bfloat162_rn(acc.x, acc.y), h1 = __floats2bfloat162_rn(acc.z, acc.w);
        uint2 w;
        w.x = *reinterpret_cast<const uint32_t *>(&h0);
        w.y = *reinterpret_cast<const uint32_t *>(&h1);
        reinterpret_cast<uint2 *>(a.out + (row0 + hh) * D)[d4] = w;
    }
}

int ctas_of(int num_sms) { return num_sms < kMostParts ? num_sms : kMostParts; }

int most_groups(int batch, int Nq, int per_group) {
    const long long g = (long long)Nq / per_group + batch;
    return (int)(g < Nq ? g : Nq);
}

struct Layout {
    size_t groups, gunits, gbase, cta_t, cta_g, n_groups, part_o, part_rho, part_l, bytes;
};

Layout layout_of(int batch, int Nq, int H, int D, int G) {
    const int ng = most_groups(batch, Nq, kCols / H);
    Layout l;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) & ~size_t(255);
        return at;
    };
    l.groups = take(sizeof(Group) * (size_t)ng);
    l.gunits = take(8 * ((size_t)ng + 1));
    l.gbase = take(4 * ((size_t)batch + 1));
    l.cta_t = take(8 * ((size_t)G + 1));
    l.cta_g = take(4 * (size_t)G);
    l.n_groups = take(4);
    l.part_o = take(4 * (size_t)2 * G * kCols * D);
    l.part_rho = take(4 * (size_t)2 * G * kCols);
    l.part_l = take(4 * (size_t)2 * G * kCols);
    l.bytes = off;
    return l;
}

template <int D, int SF>
cudaError_t launch_main(const SharedArgs &a, cudaStream_t s) {
    cudaError_t err = cudaFuncSetAttribute(shared_attend_kernel<D, SF>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           Cfg<D>::SMEM);
    if (err != cudaSuccess) return err;
    return launch_pdl(shared_attend_kernel<D, SF>, dim3(a.G), dim3(kThreads), (size_t)Cfg<D>::SMEM, s, a);
}

}  // namespace

size_t shared_attend_workspace_bytes(int batch, int Nq, int H, int D, int num_sms) {
    return layout_of(batch, Nq, H, D, ctas_of(num_sms)).bytes;
}

cudaError_t launch_shared_attend(const csa_cache &c, const void *q, int Nq, int H, const int32_t *q_offsets,
                                 const int32_t *q_pos, const float *join_out, const float *join_lse,
                                 float softmax_scale, void *out, float *lse, void *workspace, int num_sms,
                                 cudaStream_t s) {
    const int D = c.dim;
    const int G = ctas_of(num_sms);
    const Layout l = layout_of(c.batch, Nq, H, D, G);
    char *base = static_cast<char *>(workspace);
    SharedArgs a = {};
    a.fp4 = c.fp4;
    a.scale = c.scale;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.q_offsets = q_offsets;
    a.q_pos = q_pos;
    a.n_blocks = c.n_blocks;
    a.join_out = join_out;
    a.join_lse = join_lse;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.status = c.status;
    a.groups = reinterpret_cast<Group *>(base + l.groups);
    a.gunits = reinterpret_cast<long long *>(base + l.gunits);
    a.gbase = reinterpret_cast<int *>(base + l.gbase);
    a.cta_t = reinterpret_cast<long long *>(base + l.cta_t);
    a.cta_g = reinterpret_cast<int *>(base + l.cta_g);
    a.n_groups = reinterpret_cast<int *>(base + l.n_groups);
    a.part_o = reinterpret_cast<float *>(base + l.part_o);
    a.part_rho = reinterpret_cast<float *>(base + l.part_rho);
    a.part_l = reinterpret_cast<float *>(base + l.part_l);
    a.batch = c.batch;
    a.cap = c.capacity;
    a.m = c.block;
    a.Nq = Nq;
    a.H = H;
    a.per_group = kCols / H;
    a.G = G;
    a.groups_max = most_groups(c.batch, Nq, a.per_group);
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    shared_schedule_kernel<<<1, 1024, 0, s>>>(a);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const bool e4m3 = c.scale_fmt == CSA_SCALE_E4M3_16;
    if (D == 512) err = e4m3 ? launch_main<512, kScaleE4M3x16>(a, s) : launch_main<512, kScaleE8M0x32>(a, s);
    else err = e4m3 ? launch_main<128, kScaleE4M3x16>(a, s) : launch_main<128, kScaleE8M0x32>(a, s);
    if (err != cudaSuccess) return err;
    if (G < 2) return cudaSuccess;
    return launch_pdl(shared_merge_kernel, dim3(G - 1, kCols / kMergeCols, D / 128), dim3(256), 0, s, a, D);
}

}  // namespace csa
