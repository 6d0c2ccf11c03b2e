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
// 128 blocks is so dequantized once per 64 / H queries: with 64 heads once a query, as in
// attend.cu, and queries of one slot then share only its blocks' way into L2. Head counts
// that do not divide 64 leave columns empty (24 of them at 40 heads: 512 x 40 heads over
// 16384 blocks take 1.41 ms, as 64 do). Group = up to 64 columns; the flat list of all groups'
// tiles is cut into one range per CTA by cost, and groups that several CTAs share
// leave unnormalised partials for shared_merge_kernel.
//
// The products are transposed, as in attend.cu, because O of 64 columns x 512
// channels fills half of an SM's tensor memory in float32: S^T = E' Q'^T (M = 128
// blocks, N = 64 columns), O^T += E'^T P' (M = 128 channels, N = 64, K = 128 blocks).
// Operands are fp16: E'_j = e_j 2^-R_j and q' = q 2^-sQ are exact (R_j: the row's
// largest E8M0 exponent, 7 with E4M3 scales; sQ puts each column's max |q| into
// [2^14, 2^15), and what lies below 2^-31 of that is off by up to 2^-39 of it);
// P' = 2^(u log2 e + (R_j - B) - rho) <= 2^15, with B a common exponent, is
// rounded to fp16's 11 bits, which leaves about 1e-4 of the output's norm, an order
// below the bf16 rounding of the output. References rho lie 7 bits below the largest logit that
// they were taken from, so that a weight loses bits only below 2^-21 of the largest one, and all of them
// below 2^-32: what n such blocks are short of together is n 2^-32 of the output (2^-13 at 2^19 blocks; with
// references at the largest logit it was 2^-25 a block, 0.8% at 2^18). Row sums, references and accumulators are
// float32.
//
// Warp roles (20 warps, one CTA per SM): eight dequantize (they also bring the group's queries in), eight do the
// softmax and the outputs, two prepare the rows' exponents and scale factors a tile ahead, one thread each issues
// the MMAs of S^T and of O^T. At D = 512 a tile of E' takes 128 KB of shared memory, which leaves no room for a
// second one of 128 blocks (two of 64 have not been tried): a part (128 channels) of the next tile is dequantized as
// soon as O^T has read that part of this one,
// and S^T follows part by part. At D = 128 three tiles fit.
//
// What bounds it: the chain S^T -> softmax -> O^T -> dequantization of the freed parts. Measured at D = 512, 64
// heads: a tile of 64 columns takes about 5600 cycles, of which S^T's last part 420, the softmax to the last warp's
// P' 1950 (512 of them exponentials, at 16 a cycle), O^T's first part 500 and the dequantization of two parts by
// each team 2100, with a few hundred for each hand-over. (The last is bound by issue rather than by the conversions:
// integer instructions for a quarter of them took 1.47 ms.) An MMA of M = 128, N = 64, K = 16 takes 48 cycles here
// (A's 4 KB from shared memory) against 32 at the tensor rate, so the products alone would take 3000.
// 512 queries x 64 heads over 16384 blocks, causal: 1.42 ms, 0.77 PFLOP/s.
//
// Three things that mattered more than the count of instructions. (1) The roles' loops share an instruction cache
// that they overflow easily, and misses then go to one that all SMs of a GPC share: with E' of S^T passed through
// tensor memory instead (dequantized twice, so that S^T runs beside O^T) the loops came to 47 KB, 140 lines a tile
// missed, and a tile took 6500 cycles although less of it was serial (1.58 ms). (2) With the carve-out at its
// largest every spilled register is a trip to L2 (see keep_registers). (3) O^T's 32 MMAs in one straight run go out
// every 48 cycles; a barrier and a fence between the parts, all of them long ready, made it 75 (1.61 ms).
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
constexpr int kSoftmaxWarps = 8, kDequantWarps = 8;  // the latter in two teams of four
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kThreads = 32 * (kSoftmaxWarps + kDequantWarps + 4);  // whole groups of four, which registers are split by
constexpr int kTeamWarps = 4;
constexpr int kMmaWarp = kSoftmaxWarps + kDequantWarps;  // S^T; the one behind it: O^T
constexpr int kFactorWarp = kMmaWarp + 2, kFactorWarps = 2;
// Row exponents count from B, the largest of the group's first tile in the CTA (127, that is 1, when
// its rows are all zero), or kLeastBase if that is larger. fp16 holds a row of 2^(B - 10) .. 2^(B + 12) exactly without
// an exponent of its own (groups down to 2^-13 of the row's largest, which a row at B has down to 2^-23), and then
// takes none: R = 0. Others take theirs, but at least B - kExponentSpan: what that flushes to zero lies below 2^-104 of
// the first tile's scale (none where B is kLeastBase, whose rows reach down to byte 1), and no sum leaves float32's
// range over all-zero rows (scale byte 0; 2^(15 + 80) each). With kLeastBase, factors 2^(R - B) stay in float32's
// range for rows up to byte 187 (2^60) behind a first tile of any scale, and so do their products with the columns'
// (scales beyond that: up to 2^100 times the first tile's); counted from the tile's own B, ordinary rows behind a tile
// of scale byte 1 gave NaN.
constexpr int kNoRow = 1024;  // of a row behind the last visible one: its factors come out 0
constexpr int kExponentSpan = 80, kLeastBase = kExponentSpan + 1, kEvenBelow = 10, kEvenAbove = 12;
// cost units by which the tile list is shared out: a tile, and the start of a group (its queries, its output)
constexpr long long kTileUnits = 100, kStartUnits = 150;
constexpr int kScaleE8M0x32 = 0, kScaleE4M3x16 = 1;
// P' in bits: what a column's largest logit starts at when its reference is taken, and from where on the reference is
// raised. Eight bits between them make a raise rare; fp16 ends at 2^16.
constexpr float kStartBits = 7.f, kMostBits = 15.f;
// Calls of up to so many groups and slots are planned in shared memory (2.5 instead of 5.6 us; planned by every CTA of
// the main kernel for itself, a launch less, they made that kernel's registers spill: 94 -> 106 us at 32 queries then).
constexpr int kSmallGroups = 512;
constexpr int kMostCtas = 256;

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
    static constexpr int FAC_ROW = D / 16;               // bytes of a row's factors
    static constexpr int FAC_BYTES = kTile * FAC_ROW;    // of a tile; two of them
    static constexpr int SMEM = 1024 + NBUF * E_BYTES + Q_BYTES + NP * P_BYTES + 2 * FAC_BYTES + MISC;
};

// A group of columns: queries q0 .. q0 + nq - 1 of slot b, its tiles t0 .. t0 + tiles - 1 of the flat list.
struct __align__(16) Group {
    int b, q0, nq, n_max;  // n_max / n_min: most and fewest visible blocks of its queries
    int n_min, tiles;
    long long t0;
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
    int *merge_g;              // [G] the group that a CTA's first tile lies inside of and that it is the first to, or -1
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
// Where CTA c's share of all units begins: the nearest tile boundary, and the group of the first tile from there on.
struct Share {
    long long t;
    int first;
};
template <typename T>
__device__ __forceinline__ Share share_of(const T *gunits, const Group *groups, int NG, T tiles, T units, int c, int G) {
    Share s = {(long long)tiles, max(NG - 1, 0)};
    if (c < G && NG > 0) {
        const T ub = (T)((long long)units * c / G);
        int lo = 0, hi = NG - 1;  // last group with gunits[g] <= ub
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (gunits[mid] <= ub) lo = mid; else hi = mid - 1;
        }
        const int n = groups[lo].tiles;
        const T x = ub - gunits[lo] - (T)kStartUnits;
        const int k = x > 0 ? (int)min((x + (T)kTileUnits / 2) / (T)kTileUnits, (T)n) : 0;
        s.t = groups[lo].t0 + k;
        s.first = k == n && lo + 1 < NG ? lo + 1 : lo;
    }
    return s;
}
// The group that has tiles before and behind CTA c's first one, if no CTA before c begins inside it, too; else -1.
template <typename T>
__device__ __forceinline__ int merge_of(const Group *groups, const T *cta_t, const int *cta_g, int c) {
    if (c == 0) return -1;
    const int g = cta_g[c];
    const long long t = cta_t[c], t0 = groups[g].t0;
    return t > t0 && t < t0 + groups[g].tiles && cta_t[c - 1] <= t0 ? g : -1;
}

// The record of group g of slot b (its first group gb): queries, visible blocks, tiles.
__device__ __forceinline__ Group group_of(const SharedArgs &a, int b, int first) {
    Group r = {};
    r.b = b;
    r.q0 = query_bound(a, b) + first * a.per_group;
    r.nq = min(a.per_group, query_bound(a, b + 1) - r.q0);
    r.n_min = 0x7fffffff;
    for (int k = 0; k < r.nq; ++k) {
        const int n = visible_of(a, b, r.q0 + k);
        r.n_max = max(r.n_max, n);
        r.n_min = min(r.n_min, n);
    }
    r.tiles = max(1, (r.n_max + kTile - 1) / kTile);
    return r;
}
__device__ __forceinline__ int groups_in(const SharedArgs &a, int b) {
    return (max(query_bound(a, b + 1) - query_bound(a, b), 0) + a.per_group - 1) / a.per_group;
}

// The plan of a call of at most kSmallGroups groups and slots: the same steps, on shared memory.
__global__ void __launch_bounds__(kSmallGroups) shared_plan_kernel(SharedArgs a) {
    __shared__ int tmp[32], gbase[kSmallGroups + 1], gunits[kSmallGroups + 1], cta_t[kMostCtas + 1], cta_g[kMostCtas];
    __shared__ Group tab[kSmallGroups];
    const int tid = threadIdx.x;
    grid_dep_launch();
    const int mine = tid < a.batch ? groups_in(a, tid) : 0;
    const int before = block_inclusive_scan<int>(mine, tmp);
    if (tid < a.batch) gbase[tid + 1] = min(before, kSmallGroups);
    if (tid == 0) gbase[0] = 0;
    __syncthreads();
    const int NG = min(gbase[a.batch], a.groups_max);  // (groups_max only cuts offsets that are not ascending)
    Group r = {};
    if (tid < NG) {
        int lo = 0, hi = a.batch - 1;  // the slot with gbase[b] <= g < gbase[b + 1]
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (gbase[mid + 1] <= tid) lo = mid + 1; else hi = mid;
        }
        r = group_of(a, lo, tid - gbase[lo]);
    }
    const int units = tid < NG ? (int)(kStartUnits + kTileUnits * r.tiles) : 0;
    const int tin = block_inclusive_scan<int>(r.tiles, tmp), uin = block_inclusive_scan<int>(units, tmp);
    if (tid < NG) {
        r.t0 = tin - r.tiles;
        tab[tid] = r;
        a.groups[tid] = r;
        gunits[tid + 1] = uin;
    }
    if (tid == 0) gunits[0] = 0;
    if (tid == blockDim.x - 1) {
        tmp[0] = tin;
        tmp[1] = uin;
    }
    __syncthreads();
    const int tiles_all = tmp[0], units_all = tmp[1];
    for (int c = tid; c <= a.G; c += blockDim.x) {
        const Share x = share_of<int>(gunits, tab, NG, tiles_all, units_all, c, a.G);
        cta_t[c] = (int)x.t;
        a.cta_t[c] = x.t;
        if (c < a.G) a.cta_g[c] = cta_g[c] = x.first;
    }
    __syncthreads();
    for (int c = tid; c < a.G; c += blockDim.x) a.merge_g[c] = NG > 0 ? merge_of(tab, cta_t, cta_g, c) : -1;
}

// ... and of any call. One thread block: groups of every slot, their tiles, and the CTAs' ranges. A group without a
// visible block keeps one (wholly masked) tile, so that its output is written like any other.
__global__ void __launch_bounds__(1024) shared_schedule_kernel(SharedArgs a) {
    __shared__ long long tmp[32];
    __shared__ long long round_total;
    grid_dep_launch();
    long long carry = 0;
    for (int base = 0; base < a.batch; base += blockDim.x) {
        const int b = base + threadIdx.x;
        const long long g = b < a.batch ? groups_in(a, b) : 0;
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
        int tiles = 0;
        long long units = 0;
        Group r = {};
        if (g < NG) {
            int lo = 0, hi = a.batch - 1;  // the slot with gbase[b] <= g < gbase[b + 1]
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (a.gbase[mid + 1] <= g) lo = mid + 1; else hi = mid;
            }
            r = group_of(a, lo, g - a.gbase[lo]);
            tiles = r.tiles;
            units = kStartUnits + kTileUnits * tiles;
        }
        const long long tin = block_inclusive_scan<long long>(tiles, tmp);
        if (g < NG) {
            r.t0 = tcarry + tin - tiles;
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
    if (threadIdx.x == 0) a.gunits[0] = 0;
    __threadfence_block();
    __syncthreads();
    // CTA c begins at the tile boundary nearest to its share of the units
    for (int c = threadIdx.x; c <= a.G; c += blockDim.x) {
        const Share x = share_of(a.gunits, a.groups, NG, tcarry, ucarry, c, a.G);
        a.cta_t[c] = x.t;
        if (c < a.G) a.cta_g[c] = x.first;
    }
    __threadfence_block();
    __syncthreads();
    for (int c = threadIdx.x; c < a.G; c += blockDim.x) a.merge_g[c] = merge_of(a.groups, a.cta_t, a.cta_g, c);
}

// ---------------------------------------------------------------- operands
// Four neighbouring lanes share a row: lane v of them takes its 32-channel group v of every part (128 channels,
// 64 bytes of codes), so that a warp's 16-byte load covers whole 64-byte pieces of eight rows.

// A load that is issued where it stands (left to itself it is moved down to its use, a part later).
__device__ __forceinline__ uint4 load_here(const uint8_t *p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

__device__ __forceinline__ uint32_t load_word(const uint8_t *p) {
    uint32_t r;
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(r) : "l"(p));
    return r;
}

// Eight E2M1 codes to four fp16 pairs. (One conversion takes any byte of a register as it is; the header's
// function for a byte value first cuts it out: 8 instead of about 14 instructions a word with the scaling.)
__device__ __forceinline__ void e2m1_halves(uint32_t w, uint32_t (&o)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
}

// Where a part's 16 chunks of 8 channels go: chunk 4 v + k (lane v's word k) becomes chunk 8 (k / 2) + 2 v + k % 2, so
// that for every k the eight lanes of two rows store to eight different banks. Outputs are read back through
// channel_at, and the queries follow in the same order.
__device__ __forceinline__ int chunk_place(int kc) { return 8 * ((kc >> 1) & 1) + 2 * (kc >> 2) + (kc & 1); }
__device__ __forceinline__ int channel_at(int pos) {  // of a part's position
    const int pc = pos >> 3;
    return 8 * (4 * ((pc & 7) >> 1) + 2 * (pc >> 3) + (pc & 1)) + (pos & 7);
}

// The factors of a lane's 32 channels of one part of a row, as fp16 pairs: of words 0 and 1, and of 2 and 3. f: the
// factor warps' 16 bits, twice.
template <int SF>
__device__ __forceinline__ void scale_halves(uint32_t f, uint32_t (&s2)[2]) {
    if constexpr (SF == kScaleE8M0x32) {
        s2[0] = s2[1] = f;
    } else {  // two scales, E' = e 2^-7
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(f & 0xFFFF), __NV_E4M3);
        const __half2 x = __hmul2(__half2(h), __halves2half2(__ushort_as_half((15 - 7) << 10), __ushort_as_half((15 - 7) << 10)));
        const uint32_t w = *reinterpret_cast<const uint32_t *>(&x);
        s2[0] = __byte_perm(w, 0, 0x1010);
        s2[1] = __byte_perm(w, 0, 0x3232);
    }
}

// 2^(X - R) of the bytes `at` of two words, as a pair of fp16 (which rounds what lies below 2^-25 to zero).
__device__ __forceinline__ uint32_t factor_pair(uint32_t lo, uint32_t hi, int at, int R) {
    const int x = max((int)((lo >> (8 * at)) & 0xFF) - R + 127, 0), y = max((int)((hi >> (8 * at)) & 0xFF) - R + 127, 0);
    const __half2 h = __floats2half2_rn(__uint_as_float((uint32_t)x << 23), __uint_as_float((uint32_t)y << 23));
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Sixteen codes to eight fp16 pairs.
__device__ __forceinline__ void scaled_halves(uint32_t w0, uint32_t w1, uint32_t s2, uint32_t (&o)[8]) {
    uint32_t x[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        e2m1_halves(k ? w1 : w0, x);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const __half2 h = __hmul2(*reinterpret_cast<const __half2 *>(&x[b]), *reinterpret_cast<const __half2 *>(&s2));
            o[4 * k + b] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
}

// Row 32 dw + rl + 8 I of a part into its place in the 128-byte-swizzled tile in shared memory. to0, to1: the places of
// words 0 and 1 of row 32 dw + rl; words 2 and 3 lie a slice further on.
template <int SF, int I, int SLICE>
__device__ __forceinline__ void dequant_smem(const uint4 &code, uint32_t f, uint32_t to0, uint32_t to1) {
    uint32_t s2[2], o[8];
    scale_halves<SF>(f, s2);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        scaled_halves(k ? code.z : code.x, k ? code.w : code.y, s2[k], o);
#pragma unroll
        for (int z = 0; z < 2; ++z)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"((z ? to1 : to0) + I * 1024 + k * SLICE), "r"(o[4 * z]),
                         "r"(o[4 * z + 1]), "r"(o[4 * z + 2]), "r"(o[4 * z + 3])
                         : "memory");
    }
}

// ---------------------------------------------------------------- main kernel
// 20 warps leave 96 registers a thread. Saying so at the start of a role changes no split, but makes the compiler
// allocate the role by itself: without it values that only rare paths need are spilled around the tile loop, and
// with nearly all of L1 taken as shared memory every reload is a trip to L2 (2.2 ms against 1.64 when it was added,
// at D = 512, 512 x 64 heads over 16384 blocks).
__device__ __forceinline__ void keep_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 96;"); }

// Two float32 at a time (one instruction for both), and 2^x to 2^-22 relative with results below 2^-126 as zero.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float pow2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A bounded wait of one thread for a barrier's phase; most find it complete.
__device__ __forceinline__ bool wait(const uint64_t *bar, uint32_t parity, const volatile int *abort) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done || mbar_wait_ab<false>(smem_u32(bar), parity, abort);
}

// One lane of the warp, the same one every time (the compiler then knows that a single thread runs).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// tcgen05.mma with descriptors given as a low word (address, leading offset) and a high one that all
// of an operand's tiles share.
__device__ __forceinline__ void mma(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                    bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}\n"
        :
        : "r"(d), "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

// Sixteen rows by 64 columns of TMEM (fragment of m8n8 matrices): v[4 b + e] is row lane / 4, v[4 b + 2 + e] row
// lane / 4 + 8, of column 8 b + 2 (lane % 4) + e.
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(r[k]);
}

// Reduction over the eight lanes with the same lane % 4 (its column pairs v[b], b = 0 .. 7): afterwards v[0] of lane
// L is the pair b = L / 4, columns 2 L and 2 L + 1 of the 64.
template <bool MAX>
__device__ __forceinline__ void reduce_columns(float2 (&v)[8]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int half = 4; half >= 1; half >>= 1) {
        const bool hi = (lane & (4 * half)) != 0;
#pragma unroll
        for (int k = 0; k < half; ++k) {
            const float2 send = hi ? v[k] : v[k + half], keep = hi ? v[k + half] : v[k];
            const float gx = __shfl_xor_sync(0xffffffffu, send.x, 4 * half);
            const float gy = __shfl_xor_sync(0xffffffffu, send.y, 4 * half);
            v[k] = MAX ? make_float2(fmaxf(keep.x, gx), fmaxf(keep.y, gy)) : make_float2(keep.x + gx, keep.y + gy);
        }
    }
}

// B + 127 from what the factor warps found (E8M0).
__device__ __forceinline__ int base_of(const int (&b)[kFactorWarps]) {
    const int m = max(b[0], b[1]);
    return m > 0 ? max(m, kLeastBase) : 127;
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
        if (top != -INFINITY || other != other) {
            const float x = expf(lse - top), y = expf(other - top);
            f *= x / (x + y);
            jf = y / (x + y);
            lse = top + logf(x + y);
        }
    }
}

// Where a role stands in the CTA's range.
struct Cursor {
    int g, seg;       // group, and its number within the CTA
    int lt;           // tile within the group
    int left, mine;   // tiles left of the range, and of the group within the range (this one included)
    bool first;       // first tile of the group within the range
};

// Shared state behind the operand buffers.
struct Misc {
    uint64_t e_full[3][4], e_free[3][4], s_full[2], s_free[2], p_full[2], pv_done[2], q_full, q_free, o_free[2], r_full[2], drain[2];
    uint64_t f_full[2];
    uint32_t tmem;
    int abort;
    alignas(16) float minus_rho[kCols], alpha[kCols], fac[kCols], jfac[kCols];
    float wred[kSoftmaxWarps][kCols];
    float colmul[2][kCols];  // scale_log2 * 2^(sQ + B) of each column, by segment parity
    int nvis[2][kCols];
    float rexp[2][kTile];    // R_j - B
    int base[2][kFactorWarps];  // largest exponent byte of each factor warp's rows, by segment parity
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
    uint8_t *fac = P + C::NP * C::P_BYTES;
    Misc *ms = reinterpret_cast<Misc *>(fac + 2 * C::FAC_BYTES);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int b = 0; b < C::NBUF; ++b)
            for (int p = 0; p < C::PARTS; ++p) {
                mbar_init(smem_u32(&ms->e_full[b][p]), kTeamWarps);
                mbar_init(smem_u32(&ms->e_free[b][p]), 1);
            }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&ms->s_full[b]), 1);
            mbar_init(smem_u32(&ms->s_free[b]), kSoftmaxWarps);
            mbar_init(smem_u32(&ms->p_full[b]), kSoftmaxWarps);
            mbar_init(smem_u32(&ms->pv_done[b]), 1);
            mbar_init(smem_u32(&ms->o_free[b]), kSoftmaxWarps);
            mbar_init(smem_u32(&ms->f_full[b]), kFactorWarps);
            mbar_init(smem_u32(&ms->r_full[b]), kFactorWarps);
            mbar_init(smem_u32(&ms->drain[b]), 1);
        }
        mbar_init(smem_u32(&ms->q_full), kDequantWarps);
        mbar_init(smem_u32(&ms->q_free), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        ms->abort = 0;
    }
    if (tid < kCols) ms->minus_rho[tid] = 0.f;
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
    const long long t_begin = a.cta_t[blockIdx.x];
    const int n_tiles = (int)(a.cta_t[blockIdx.x + 1] - t_begin);
    auto start = [&]() {
        Cursor c;
        c.g = a.cta_g[blockIdx.x];
        c.seg = 0;
        c.lt = (int)(t_begin - a.groups[c.g].t0);
        c.left = n_tiles;
        c.mine = min(c.left, a.groups[c.g].tiles - c.lt);
        c.first = true;
        return c;
    };
    // the next tile (the caller checks c.left > 0)
    auto step = [&](Cursor &c) {
        ++c.lt;
        --c.left;
        --c.mine;
        c.first = false;
        if (c.mine == 0 && c.left > 0) {
            ++c.g;
            ++c.seg;
            c.lt = 0;
            c.mine = min(c.left, a.groups[c.g].tiles);
            c.first = true;
        }
    };

    if (n_tiles <= 0) {
        // nothing to do: fall through to the common end
    } else if (warp < kSoftmaxWarps) {
        // ================================================================ softmax and output
        keep_registers();
        // S^T: 16 rows (blocks) a warp, and of them two a thread, in all 64 columns of which a thread has 16:
        // rows r0 and r0 + 8, columns 8 b + 2 (lane % 4) + {0, 1}, b = 0 .. 7 (the fragment that 16x256b loads
        // give and stmatrix takes). A column's factors are so read once for two rows.
        // O^T: 32 lanes (channels) and 32 columns a warp, one channel a thread.
        const int hf = tid >> 7, r0 = 32 * (warp & 3) + 16 * hf + (lane >> 2), c0 = 2 * (lane & 3);
        const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t s_addr = tmem + lane_off + ((uint32_t)(16 * hf) << 16);
        const uint32_t o_addr = tmem + lane_off + C::TMEM_O + 32 * hf;
        // stmatrix: lanes 8 i .. 8 i + 7 address matrix i = (rows 0-7 | 8-15) of column blocks b and b + 1
        const uint32_t p_addr = smem_u32(P) + (4 * (warp & 3) + 2 * hf + ((lane >> 3) & 1)) * 1024 + (lane & 7) * 128 +
                                (((lane >> 4) ^ (lane & 7)) << 4);
        float2 lsum[8];  // sums of this thread's columns over its rows
        int n = 0;       // tiles done by this CTA
        Cursor c = start();
        while (c.left > 0) {
            const int n_min = a.groups[c.g].n_min, mp = c.seg & 1;
            const bool from_start = c.lt == 0;
            bool gave_up = false, ok = true;
#pragma unroll
            for (int b = 0; b < 8; ++b) lsum[b] = make_float2(0.f, 0.f);
            while (true) {
                const bool first = c.first;
                const int sb = n & 1;
                // the rows' exponents from B on: 0 for almost all of them
                ok = ok && wait(&ms->f_full[sb], (n >> 1) & 1, abort);
                const float R0 = ms->rexp[sb][r0], R1 = ms->rexp[sb][r0 + 8];
                const bool even = !__any_sync(0xffffffffu, R0 != 0.f || R1 != 0.f);
                const bool masked = (c.lt + 1) * kTile > n_min;
                ok = ok && wait(&ms->s_full[sb], (n >> 1) & 1, abort);
                tc_fence_after();
                float u[32];
                // u + R - rho of this thread's rows and columns. References are set by the group's first tile, and
                // raised (with O^T and the sums) when a logit exceeds one by more than kMostBits: then once more from
                // the start, with the new ones. (A second raise happens only where a logit is so large that
                // the first one was rounded; what rounding then leaves above is cut.) A wait that ran out
                // comes this way too.
                for (int pass = 0;; ++pass) {
                    float over = -INFINITY;
                    tmem_ld_rows(s_addr + kCols * sb, u);
                    if (even) {
#pragma unroll
                        for (int b = 0; b < 8; ++b) {
                            const float2 cm = *reinterpret_cast<const float2 *>(&ms->colmul[mp][8 * b + c0]);
                            const float2 rh = *reinterpret_cast<const float2 *>(&ms->minus_rho[8 * b + c0]);
                            const float2 x = fma2(make_float2(u[4 * b], u[4 * b + 1]), cm, rh);
                            const float2 y = fma2(make_float2(u[4 * b + 2], u[4 * b + 3]), cm, rh);
                            u[4 * b] = x.x;
                            u[4 * b + 1] = x.y;
                            u[4 * b + 2] = y.x;
                            u[4 * b + 3] = y.y;
                        }
                    } else {
                        const float m0 = pow2(R0), m1 = pow2(R1);
#pragma unroll
                        for (int b = 0; b < 8; ++b) {
                            const float2 cm = *reinterpret_cast<const float2 *>(&ms->colmul[mp][8 * b + c0]);
                            const float2 rh = *reinterpret_cast<const float2 *>(&ms->minus_rho[8 * b + c0]);
                            u[4 * b] = fmaf(u[4 * b], cm.x * m0, rh.x + R0);
                            u[4 * b + 1] = fmaf(u[4 * b + 1], cm.y * m0, rh.y + R0);
                            u[4 * b + 2] = fmaf(u[4 * b + 2], cm.x * m1, rh.x + R1);
                            u[4 * b + 3] = fmaf(u[4 * b + 3], cm.y * m1, rh.y + R1);
                        }
                    }
                    if (masked) {
                        const int e0 = c.lt * kTile + r0;
#pragma unroll
                        for (int b = 0; b < 8; ++b) {
                            const int2 nv = *reinterpret_cast<const int2 *>(&ms->nvis[mp][8 * b + c0]);
                            if (e0 >= nv.x) u[4 * b] = -INFINITY;
                            if (e0 >= nv.y) u[4 * b + 1] = -INFINITY;
                            if (e0 + 8 >= nv.x) u[4 * b + 2] = -INFINITY;
                            if (e0 + 8 >= nv.y) u[4 * b + 3] = -INFINITY;
                        }
                    }
                    if (pass >= 2) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) u[k] = u[k] > kMostBits ? kMostBits : u[k];
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) over = fmaxf(over, fmaxf(fmaxf(u[k], u[k + 8]), fmaxf(u[k + 16], u[k + 24])));
                    const bool set = first && pass == 0;
                    if (!bar_or_n<kSoftmaxThreads>(set || over > kMostBits || !ok)) break;
                    if (!first) ok = ok && wait(&ms->pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, abort);
                    float2 m[8];
#pragma unroll
                    for (int b = 0; b < 8; ++b)
                        m[b] = make_float2(fmaxf(u[4 * b], u[4 * b + 2]), fmaxf(u[4 * b + 1], u[4 * b + 3]));
                    reduce_columns<true>(m);  // lane L: columns 2 L and 2 L + 1
                    *reinterpret_cast<float2 *>(&ms->wred[warp][2 * lane]) = m[0];
                    if (bar_or_n<kSoftmaxThreads>(!ok)) {
                        ms->abort = 1;
                        gave_up = true;
                        break;
                    }
                    if (tid < kCols) {
                        float M = ms->wred[0][tid];
#pragma unroll
                        for (int w = 1; w < kSoftmaxWarps; ++w) M = fmaxf(M, ms->wred[w][tid]);
                        // (a column that sees nothing of its first tile sees nothing of the others)
                        const bool raise = set ? M > -INFINITY : M > kMostBits;
                        if (raise) ms->minus_rho[tid] -= M - kStartBits;
                        ms->alpha[tid] = raise ? pow2(kStartBits - M) : 1.f;
                    }
                    bar_sync_n<kSoftmaxThreads>();
                    if (!first) {
                        tc_fence_after();
#pragma unroll 1
                        for (int x = 0; x < 2 * C::PARTS; ++x) {
                            float o[16];
                            const uint32_t at = o_addr + kCols * (x >> 1) + 16 * (x & 1);
                            tmem_ld16(at, o);
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] *= ms->alpha[32 * hf + 16 * (x & 1) + k];
                            tmem_st16(at, o);
                        }
#pragma unroll
                        for (int b = 0; b < 8; ++b)
                            lsum[b] = mul2(lsum[b], *reinterpret_cast<const float2 *>(&ms->alpha[8 * b + c0]));
                    }
                }
                if (gave_up) break;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ms->s_free[sb]));
                // P' = 2^(u - rho), fp16
                const uint32_t Pn = p_addr + (n % C::NP) * C::P_BYTES;
#pragma unroll
                for (int k = 0; k < 32; ++k) u[k] = pow2(u[k]);
                if (n >= C::NP)  // P' is free: the O^T product of tile n - NP is done (a failure shows in the next vote)
                    ok = wait(&ms->pv_done[(n - C::NP) & 1], ((n - C::NP) >> 1) & 1, abort) && ok;
#pragma unroll
                for (int b = 0; b < 8; b += 2) {
                    uint32_t pk[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int k = 4 * b + 2 * q;
                        const __half2 hh = __floats2half2_rn(u[k], u[k + 1]);
                        pk[q] = *reinterpret_cast<const uint32_t *>(&hh);
                    }
                    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(Pn ^ (b << 4)),
                                 "r"(pk[0]), "r"(pk[1]), "r"(pk[2]), "r"(pk[3])
                                 : "memory");
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
#ifdef CSA_TEST_LOST_WEIGHTS  // a test build in which O^T waits in vain for the last tile's weights
                if (lane == 0 && !(warp == 0 && c.left == 1))
#else
                if (lane == 0)
#endif
                    mbar_arrive(smem_u32(&ms->p_full[n % C::NP]));
                // the sums (without 2^R, which P' carries for E'), while the O^T product runs
                if (even) {
#pragma unroll
                    for (int b = 0; b < 8; ++b)
                        lsum[b] = add2(lsum[b], add2(make_float2(u[4 * b], u[4 * b + 1]), make_float2(u[4 * b + 2], u[4 * b + 3])));
                } else {
                    const float2 i0 = make_float2(pow2(-R0), pow2(-R0)), i1 = make_float2(pow2(-R1), pow2(-R1));
#pragma unroll
                    for (int b = 0; b < 8; ++b)
                        lsum[b] = fma2(make_float2(u[4 * b], u[4 * b + 1]), i0,
                                       fma2(make_float2(u[4 * b + 2], u[4 * b + 3]), i1, lsum[b]));
                }
                ++n;
                if (c.mine == 1) break;
                step(c);
            }
            if (gave_up) break;
            // ---------------- the group's output, or its partial
            reduce_columns<false>(lsum);
            *reinterpret_cast<float2 *>(&ms->wred[warp][2 * lane]) = lsum[0];
            ok = wait(&ms->pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, abort) && ok;
            if (bar_or_n<kSoftmaxThreads>(!ok)) {
                ms->abort = 1;
                break;
            }
            const Group gr = a.groups[c.g];
            const int seg = c.seg;
            const bool whole = from_start && c.lt + 1 == gr.tiles;
            const int cols = gr.nq * a.H;
            const size_t row0 = (size_t)gr.q0 * a.H;
            // O^T holds E' = e 2^-(R - B) times P' over 2^B
            const float unit = SF == kScaleE8M0x32 ? exp2f((float)(base_of(ms->base[mp]) - 127)) : exp2f(7.f);
            const int slot = 2 * blockIdx.x + (seg == 0 ? 0 : 1);
            if (tid < kCols) {
                float l = 0.f;
#pragma unroll
                for (int w = 0; w < kSoftmaxWarps; ++w) l += ms->wred[w][tid];
                const float rho = -ms->minus_rho[tid];
                if (!whole) {
                    a.part_rho[(size_t)slot * kCols + tid] = l == 0.f ? -INFINITY : rho;
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
            for (int x = 0; x < 2 * C::PARTS; ++x) {  // 128 channels, 16 columns
                float o[16];
                const int col0 = 32 * hf + 16 * (x & 1), ch = 128 * (x >> 1) + channel_at(32 * (warp & 3) + lane);
                tmem_ld16(o_addr + kCols * (x >> 1) + 16 * (x & 1), o);
                if (x == 2 * C::PARTS - 1) {  // O^T is read: the next group's products may start
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&ms->o_free[seg & 1]));
                }
                if (!whole) {
                    float *dst = a.part_o + ((size_t)slot * kCols + col0) * D + ch;
#pragma unroll
                    for (int k = 0; k < 16; ++k) dst[(size_t)k * D] = o[k] * unit;
                } else {
                    const float *jo = a.join_out + (row0 + col0) * D + ch;
                    __nv_bfloat16 *dst = a.out + (row0 + col0 + (lane & 1)) * D + (ch & ~1);
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        float v[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int col = col0 + k + e;
                            const float f = ms->fac[col];
                            // (a NaN goes on; f * unit alone may lie below float32's range)
                            v[e] = f == 0.f ? 0.f : o[k + e] * f * unit;
                            if (a.join_lse && col < cols && ms->jfac[col] != 0.f)
                                v[e] = fmaf(ms->jfac[col], jo[(size_t)(k + e) * D], v[e]);
                        }
                        // even lanes take column k, odd ones k + 1, with their neighbour's channel
                        const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? v[0] : v[1], 1);
                        if (col0 + k + (lane & 1) < cols)
                            *reinterpret_cast<__nv_bfloat162 *>(dst + (size_t)k * D) =
                                (lane & 1) ? __floats2bfloat162_rn(got, v[1]) : __floats2bfloat162_rn(v[0], got);
                    }
                }
            }
            if (tid < kCols) ms->minus_rho[tid] = 0.f;
            bar_sync_n<kSoftmaxThreads>();  // minus_rho, fac, wred belong to the next group from here on
            step(c);
        }
    } else if (warp < kMmaWarp) {
        // ================================================================ dequantization, queries
        keep_registers();
        // Two teams of four warps. D = 512: each takes every other part of a tile; D = 128: every other tile.
        const int dw = warp & 3, team = (warp - kSoftmaxWarps) >> 2, v = lane & 3, rl = lane >> 2;
        // this lane's rows of a tile are 32 dw + rl + 8 i, i = 0 .. 3
        const int j = 32 * dw + rl;
        const uint32_t place = smem_u32(E) + j * 128;
        const uint32_t off0 = place + (((2 * v) ^ rl) << 4), off1 = place + (((2 * v + 1) ^ rl) << 4);
        constexpr int MINE = D == 512 ? 2 : 1;  // parts of a team; their codes of the team's next tile wait in registers
        Cursor c = start();
        int slot_g = c.g, slot = a.groups[c.g].b, n_max = a.groups[c.g].n_max;  // the group of the rows asked for last
        uint4 code[MINE][4];
        // this lane's first row of a tile (its codes of part 0), and how many rows from there on are visible
        // (the others are zero codes)
        struct Rows {
            const uint8_t *codes;
            int live;
        };
        auto rows_of = [&](const Cursor &x) {
            if (x.g != slot_g) {
                slot_g = x.g;
                slot = a.groups[slot_g].b;
                n_max = a.groups[slot_g].n_max;
            }
            const int e = x.lt * kTile + j;
            Rows r;
            r.codes = a.fp4 + ((size_t)slot * a.cap + e) * (D / 2) + v * 16;
            r.live = n_max - e;
            return r;
        };
        // (rows behind the last visible one load that one again; their factors are 0)
        auto load_codes = [&](uint4 (&to)[4], const uint8_t *src, int live) {
#pragma unroll
            for (int i = 0; i < 4; ++i) to[i] = load_here(src + min(8 * i, live - 1) * (D / 2));
        };
        auto part = [&](int m) { return D == 512 ? team + 2 * m : 0; };
        auto load_part = [&](int m, const Rows &r) {  // (nothing of a group without visible blocks, or behind the last tile)
            if (r.codes && n_max > 0) load_codes(code[m], r.codes + part(m) * 64, r.live);
        };
#pragma unroll
        for (int m = 0; m < MINE; ++m) {
#pragma unroll
            for (int i = 0; i < 4; ++i) code[m][i] = make_uint4(0, 0, 0, 0);
            Cursor x = c;
            if (D == 128 && team == 1) step(x);
            if (x.left > 0) load_part(m, rows_of(x));
        }
        int n = 0;
        bool ok = true;
        while (c.left > 0) {
            if (c.first) {
                const Group gr = a.groups[c.g];
                // the queries of the group: column = row q0 * H + column of q; per column 2^-sQ
                if (c.seg >= 1) ok = wait(&ms->q_free, (c.seg - 1) & 1, abort);
                if (c.seg >= 2) ok = ok && wait(&ms->o_free[c.seg & 1], ((c.seg - 2) >> 1) & 1, abort);
                if (!__all_sync(0xffffffffu, ok)) break;
                const int cols = gr.nq * a.H, mp = c.seg & 1;
                int base = 127 + 7;
                if constexpr (SF == kScaleE8M0x32) {
                    ok = wait(&ms->r_full[mp], (c.seg >> 1) & 1, abort);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    base = base_of(ms->base[mp]);
                }
                constexpr int LANES = D == 512 ? 32 : 16;      // lanes of a column
                constexpr int PER = 32 / LANES;                // columns of a warp at a time
                constexpr int CH = D / 8 / LANES;              // 16-byte chunks of a lane
                const int sub = lane / LANES, sl = lane % LANES;
#pragma unroll 1
                for (int k0 = 0; k0 < kCols / kDequantWarps; k0 += 2 * PER) {
                    uint4 v[2][CH];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int col = (warp - kSoftmaxWarps) * (kCols / kDequantWarps) + k0 + x * PER + sub;
                        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + ((size_t)gr.q0 * a.H + col) * D);
#pragma unroll
                        for (int y = 0; y < CH; ++y)
                            v[x][y] = col < cols ? __ldg(src + sl + y * LANES) : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int col = (warp - kSoftmaxWarps) * (kCols / kDequantWarps) + k0 + x * PER + sub;
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
                            const int pc = (kc & ~15) + chunk_place(kc & 15);
                            *reinterpret_cast<uint4 *>(Q + (pc >> 3) * C::QSLICE + (col >> 3) * 1024 + (col & 7) * 128 +
                                                       (((pc & 7) ^ (col & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                        if (sl == 0) {
                            ms->colmul[mp][col] = ldexpf(a.scale_log2, sq + base - 127);
                            ms->nvis[mp][col] = col < cols ? visible_of(a, gr.b, gr.q0 + col / a.H) : 0;
                        }
                    }
                }
                fence_async_smem();
                __syncwarp();
#ifdef CSA_TEST_LOST_ARRIVALS  // a test build in which nothing completes the first wait for the queries
                if (lane == 0 && warp != kSoftmaxWarps)
#else
                if (lane == 0)
#endif
                    mbar_arrive(smem_u32(&ms->q_full));
            }
            const int buf = n % C::NBUF, use = n / C::NBUF;
            if (D == 128 && (n & 1) != team) {
                step(c);
                ++n;
                continue;
            }
            // this lane's factors of the tile: 16 bits for each part
            uint2 f[4];
            ok = wait(&ms->f_full[n & 1], (n >> 1) & 1, abort) && ok;
            const uint8_t *src = fac + (n & 1) * C::FAC_BYTES + j * C::FAC_ROW + v * (C::FAC_ROW / 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (D == 512) f[i] = *reinterpret_cast<const uint2 *>(src + 8 * i * C::FAC_ROW);
                else f[i].x = *reinterpret_cast<const uint16_t *>(src + 8 * i * C::FAC_ROW);
            }
            step(c);
            Cursor x = c;  // the team's next tile
            if (D == 128 && x.left > 0) step(x);
            Rows rows = {};
            if (x.left > 0) rows = rows_of(x);
#pragma unroll
            for (int m = 0; m < MINE; ++m) {
                const int p = part(m);
                if (use >= 1) ok = wait(&ms->e_free[buf][p], (use - 1) & 1, abort) && ok;
                const uint32_t at = buf * C::E_BYTES + p * (2 * C::SLICE);
                auto factor = [&](int i) { return __byte_perm(p & 2 ? f[i].y : f[i].x, 0, p & 1 ? 0x3232 : 0x1010); };
                dequant_smem<SF, 0, C::SLICE>(code[m][0], factor(0), off0 + at, off1 + at);
                dequant_smem<SF, 1, C::SLICE>(code[m][1], factor(1), off0 + at, off1 + at);
                dequant_smem<SF, 2, C::SLICE>(code[m][2], factor(2), off0 + at, off1 + at);
                dequant_smem<SF, 3, C::SLICE>(code[m][3], factor(3), off0 + at, off1 + at);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ms->e_full[buf][p]));
                load_part(m, rows);
            }
            if (!__all_sync(0xffffffffu, ok)) break;
            ++n;
        }
        if (!ok) ms->abort = 1;
    } else {
        keep_registers();
        if (warp >= kFactorWarp) {
            // ================================================================ scales
            // The tiles' scales, a row a lane: the rows' exponents R, and each group's factor (E4M3: its byte) where the lane
            // that dequantizes it finds those of all parts together: 16 bits at [row][v][part]. In warps of their own
            // they keep that work, and its registers, out of the dequantizing warps' loop.
            constexpr int W = D / (SF == kScaleE4M3x16 ? 64 : 128);  // words of a row's scales
            const int row0 = 64 * (warp - kFactorWarp) + lane;  // and row0 + 32
            Cursor c = start();
            int n = 0, base = 127 + 7;
            bool ok = true;
            while (c.left > 0) {
                const int b = a.groups[c.g].b, n_max = a.groups[c.g].n_max;
                uint32_t w[2][W];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int e = c.lt * kTile + row0 + 32 * k;
                    const uint8_t *src = a.scale + ((size_t)b * a.cap + e) * (4 * W);
#pragma unroll
                    for (int x = 0; x < W; x += 4) {
                        if constexpr (W >= 4) {
                            const uint4 u = e < n_max ? load_here(src + 4 * x) : make_uint4(0, 0, 0, 0);
                            w[k][x] = u.x;
                            w[k][x + 1] = u.y;
                            w[k][x + 2] = u.z;
                            w[k][x + 3] = u.w;
                        } else {
#pragma unroll
                            for (int y = 0; y < W; ++y) w[k][y] = e < n_max ? load_word(src + 4 * y) : 0;
                        }
                    }
                }
                // the exponents and factors of tile n - 2 are read: its S^T, which takes all of its dequantized rows, is, too
                if (n >= 2) ok = wait(&ms->s_free[n & 1], ((n >> 1) - 1) & 1, abort) && ok;
                int m[2];  // the rows' largest exponents
                if constexpr (SF == kScaleE8M0x32) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t x = w[k][0];
#pragma unroll
                        for (int y = 1; y < W; ++y) x = __vmaxu4(x, w[k][y]);
                        x = __vmaxu4(x, x >> 16);
                        m[k] = (int)max(x & 0xFF, (x >> 8) & 0xFF);
                    }
                    if (c.first) {  // B
                        if (c.seg >= 2) ok = wait(&ms->o_free[c.seg & 1], ((c.seg - 2) >> 1) & 1, abort) && ok;
                        const int mine = __reduce_max_sync(0xffffffffu, max(m[0], m[1]));
                        if (lane == 0) {
                            ms->base[c.seg & 1][warp - kFactorWarp] = mine;
                            mbar_arrive(smem_u32(&ms->r_full[c.seg & 1]));
                        }
                        ok = wait(&ms->r_full[c.seg & 1], (c.seg >> 1) & 1, abort) && ok;
                        base = base_of(ms->base[c.seg & 1]);
                    }
                }
                if (!__all_sync(0xffffffffu, ok)) break;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int row = row0 + 32 * k;
                    uint32_t o[D == 512 ? 8 : 2];
                    int R = base;
                    if constexpr (SF == kScaleE8M0x32) {
                        const int d = m[k] - base;
                        if (d < -kEvenBelow || d > kEvenAbove) R = max(m[k], base - kExponentSpan);
                        const bool live = c.lt * kTile + row < n_max;
                        ms->rexp[n & 1][row] = live ? (float)(R - base) : 0.f;
                        if (!live) R = kNoRow;
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            if constexpr (D == 512) {
                                o[2 * v] = factor_pair(w[k][0], w[k][1], v, R);
                                o[2 * v + 1] = factor_pair(w[k][2], w[k][3], v, R);
                            } else if (v % 2 == 0) {
                                o[v / 2] = factor_pair(w[k][0] >> (8 * v), w[k][0] >> (8 * v + 8), 0, R);
                            }
                        }
                    } else {
                        ms->rexp[n & 1][row] = 0.f;
                        if constexpr (D == 512) {
#pragma unroll
                            for (int v = 0; v < 4; ++v) {
                                const uint32_t pick = v & 1 ? 0x7632 : 0x5410;
                                o[2 * v] = __byte_perm(w[k][v >> 1], w[k][2 + (v >> 1)], pick);
                                o[2 * v + 1] = __byte_perm(w[k][4 + (v >> 1)], w[k][6 + (v >> 1)], pick);
                            }
                        } else {
                            o[0] = w[k][0];
                            o[1] = w[k][1];
                        }
                    }
                    uint8_t *dst = fac + (n & 1) * C::FAC_BYTES + row * C::FAC_ROW;
                    if constexpr (D == 512) {
                        *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4 *>(dst + 16) = make_uint4(o[4], o[5], o[6], o[7]);
                    } else {
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(o[0], o[1]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ms->f_full[n & 1]));
                step(c);
                ++n;
            }
            if (!ok) ms->abort = 1;
        } else if (elect_one()) {  // (the warp's other lanes wait at the common end)
            // ================================================================ MMA issue
            // One warp issues S^T, the other O^T: either product waits for barriers of its own.
            constexpr uint32_t IDESC_S = idesc_f16(kTile, kCols, false, false);
            constexpr uint32_t IDESC_O = idesc_f16(kTile, kCols, true, true);
            const bool scores = warp == kMmaWarp;  // ... and not O^T
            // its group, the group's number within the CTA, tiles left of it
            int g = a.cta_g[blockIdx.x], seg = 0;
            int mine = min(n_tiles, (int)(a.groups[g].t0 + a.groups[g].tiles - t_begin));
            bool first = true, ok = true;  // first tile of the group within the CTA
            auto next_tile = [&](int n) {
                first = false;
                if (--mine == 0 && n + 1 < n_tiles) {
                    ++g;
                    ++seg;
                    mine = min(n_tiles - n - 1, a.groups[g].tiles);
                    first = true;
                }
            };
            if (scores) {  // E' and Q' by channels; 16 bytes a unit
                const uint64_t de = desc_sw128(smem_u32(E), 16, 1024), dq = desc_sw128(smem_u32(Q), 16, 1024);
                const uint32_t e_hi = (uint32_t)(de >> 32), q_hi = (uint32_t)(dq >> 32);
                for (int n = 0; n < n_tiles && ok; ++n) {
                    const int buf = n % C::NBUF, sb = n & 1;
                    const uint32_t d = tmem + kCols * sb;
                    if (first) ok = wait(&ms->q_full, seg & 1, abort);
                    if (n >= 2) ok = ok && wait(&ms->s_free[sb], ((n >> 1) - 1) & 1, abort);
#pragma unroll 1
                    for (int p = 0; p < C::PARTS; ++p) {
                        ok = ok && wait(&ms->e_full[buf][p], (n / C::NBUF) & 1, abort);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t a_lo = (uint32_t)de + ((buf * C::E_BYTES + p * 2 * C::SLICE) >> 4);
                        const uint32_t b_lo = (uint32_t)dq + (p * 2 * C::QSLICE >> 4);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {  // 16 channels each, 64 of a slice
                            const uint32_t b_at = b_lo + (((kk >> 2) * C::QSLICE + (kk & 3) * 32) >> 4);
                            mma(d, a_lo + (((kk >> 2) * C::SLICE + (kk & 3) * 32) >> 4), e_hi, b_at, q_hi, IDESC_S, kk > 0 || p > 0);
                        }
                    }
                    if (!ok) break;
                    mma_commit(smem_u32(&ms->s_full[sb]));
                    if (mine == 1) mma_commit(smem_u32(&ms->q_free));
                    next_tile(n);
                }
            } else {  // E' and P' by blocks
                const uint64_t dv = desc_sw128(smem_u32(E), C::SLICE, 1024), dp = desc_sw128(smem_u32(P), 8192, 1024);
                const uint32_t v_hi = (uint32_t)(dv >> 32), p_hi = (uint32_t)(dp >> 32);
                for (int n = 0; n < n_tiles && ok; ++n) {
                    const int buf = n % C::NBUF;
                    const uint32_t b_lo = (uint32_t)dp + (n % C::NP) * (C::P_BYTES >> 4);
                    ok = wait(&ms->p_full[n % C::NP], (n / C::NP) & 1, abort);
                    if (first && seg > 0) ok = ok && wait(&ms->o_free[(seg - 1) & 1], ((seg - 1) >> 1) & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int p = 0; p < C::PARTS; ++p) {  // (all parts are there: S^T read them)
                        const uint32_t a_lo = (uint32_t)dv + ((buf * C::E_BYTES + p * 2 * C::SLICE) >> 4);
#pragma unroll
                        for (int kj = 0; kj < kTile / 16; ++kj)  // 16 blocks each
                            mma(tmem + C::TMEM_O + kCols * p, a_lo + (kj * 2048 >> 4), v_hi, b_lo + (kj * 2048 >> 4), p_hi, IDESC_O,
                                kj > 0 || !first);
                        mma_commit(smem_u32(&ms->e_free[buf][p]));
                    }
                    mma_commit(smem_u32(&ms->pv_done[n & 1]));
                    next_tile(n);
                }
            }
            // Nothing issued may still run when the CTA leaves, and others may give up after this thread's last product
            // has gone out. (Otherwise they wait for it themselves: this costs nothing.)
            mma_commit(smem_u32(&ms->drain[scores]));
            if (!mbar_wait_for(smem_u32(&ms->drain[scores]), 0, kDrainCycles) || !ok) ms->abort = 1;
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
constexpr int kMergeCols = 8, kMostParts = kMostCtas;

__global__ void __launch_bounds__(256) shared_merge_kernel(SharedArgs a, int D) {
    __shared__ int slots[kMostParts];
    __shared__ float wts[kMostParts * kMergeCols];
    __shared__ float s_join[kMergeCols];
    __shared__ int np_s;
    grid_dep_wait();
    const int c = blockIdx.x + 1, g = a.merge_g[c];
    if (g < 0) return;
    const Group gr = a.groups[g];
    const long long t1 = gr.t0 + gr.tiles;
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
                has = rb < a.cta_t[cc + 1] && rb < t1 && a.cta_t[cc + 1] > gr.t0;
            }
            const uint32_t mask = __ballot_sync(0xffffffffu, has);
            const int pos = np + __popc(mask & ((1u << threadIdx.x) - 1u));
            if (has && pos < kMostParts) slots[pos] = 2 * cc + (rb >= gr.t0 ? 0 : 1);
            np += __popc(mask);
            if (!__any_sync(0xffffffffu, cc < a.G && rb < t1)) break;
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
            const float w = top == -INFINITY ? 0.f : exp2f(a.part_rho[at] - top);
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
    size_t groups, gunits, gbase, cta_t, cta_g, merge_g, part_o, part_rho, part_l, bytes;
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
    l.merge_g = take(4 * (size_t)G);
    l.part_o = take(4 * (size_t)2 * G * kCols * D);
    l.part_rho = take(4 * (size_t)2 * G * kCols);
    l.part_l = take(4 * (size_t)2 * G * kCols);
    l.bytes = off;
    return l;
}

template <int D, int SF>
cudaError_t launch_main(const SharedArgs &a, cudaStream_t s) {
    const cudaError_t err =
        cudaFuncSetAttribute(shared_attend_kernel<D, SF>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
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
    a.merge_g = reinterpret_cast<int *>(base + l.merge_g);
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
    if (a.batch <= kSmallGroups && a.groups_max <= kSmallGroups) shared_plan_kernel<<<1, kSmallGroups, 0, s>>>(a);
    else shared_schedule_kernel<<<1, 1024, 0, s>>>(a);
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
