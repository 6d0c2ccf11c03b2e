// cache_copy.cu -- csa_cache_copy: blocks of cache slots copied into other slots
// (fork, move), gathered by a list (compaction, in place too), cut short or freed.
//
// No arithmetic: every kept block's bytes of every plane (codes, scales, indexer
// keys, their scales) are read once and written once per destination, so the
// call is HBM-bound: 2 x 262143 blocks of 400 bytes to two slots each take 107 us
// (5.9 TB/s), 65521 listed blocks of 32 slots 300 us (5.6 TB/s; in place, with its waits,
// 440). Small calls are bound by the latency of its launches.
//
//   copy_check_kernel  (with long lists only) finds where each job's list ends: one
//                      thread block per 4096 entries. Lists of up to 4096 columns
//                      and together up to 32768 entries are read by the plan kernel,
//                      one warp a job, which saves a launch (about 4 us of a small
//                      call); a list is then one part, whose end that warp finds.
//   copy_plan_kernel   one thread block: counts, refusals, the flat list of
//                      tiles (64 blocks each) and the new n_blocks.
//   cache_move_kernel  four or more thread blocks per SM take tiles from a
//                      counter, load a tile's rows of every plane into shared
//                      memory (cp.async, 16 bytes where the addresses allow) and
//                      write them out. Jobs in a row with the same source and
//                      count share a tile: it is read once and written to up to
//                      kFan destinations.
//
// In place, tile t of a job overwrites blocks that earlier tiles of the job may
// still have to read (an ascending list moves block j to a place <= j, so never
// later ones). Every tile loads all its rows before it writes, and sets a flag in
// between; a tile writes once the tiles whose sources lie in its destination have
// set theirs -- as a rule one or two, found by searching the list while the rows
// load. Tiles are handed out in order, each thread block one ahead, and
// loading waits for nothing: of the tiles that have not loaded the first one is never
// behind a tile that still waits, so every wait ends.
#include "common.cuh"
#include "tc_util.cuh"

namespace csa {

namespace {

constexpr int kMoveThreads = 256;
constexpr int kTileRows = 64;
constexpr int kFan = 4;          // destinations that share the read of a tile
constexpr int kCheckPart = 4096; // list entries of one check block
constexpr int kPlanThreads = 1024;
constexpr int kPlanSmemBatch = 1024;
constexpr int kPlanEntries = 32768;  // list entries that the plan kernel reads itself, in lists of one part

// Shared memory of a plane's tile: its rows, and room for the tile's offset from a 16-byte boundary.
constexpr int tile_bytes(int row) { return (kTileRows * row + 15) / 16 * 16 + 16; }
// The largest tile of any admitted layout: dim 512, E4M3 scales, bf16 keys of 256 channels.
constexpr int kMostTileBytes = tile_bytes(256) + tile_bytes(32) + tile_bytes(512);

struct Plane {
    const uint8_t *src;
    uint8_t *dst;
    int row;  // bytes of a block's row
    int at;   // offset of the plane's tile in shared memory
};

// One job as the move kernel sees it (n < 0: nothing to move).
struct JobRec {
    int src, dst, n, followers;  // followers: jobs behind it that share its tiles
};

struct CopyArgs {
    Plane plane[4];
    int planes;
    int src_batch, src_cap, dst_batch, dst_cap, same;
    const int32_t *src_n;
    int32_t *dst_n;
    int32_t *status;
    const int32_t *src_slot, *dst_slot, *keep, *max_blocks;
    int jobs, cols, parts, list_tiles;
    int plan_lists;  // the plan kernel finds the lists' ends
    // workspace
    JobRec *rec;           // [jobs]
    long long *prefix;     // [jobs + 1] tiles
    unsigned long long *ticket;
    int *slot_tab;         // [3][dst_batch] when it does not fit shared memory
    int *part_end;         // [jobs][parts]: 2 * position + bad, of the part's first ending entry, or -1
    int *flags;            // [jobs][list_tiles]
};

__device__ __forceinline__ int filled(const int32_t *n, int slot, int cap) { return min(max(n[slot], 0), cap); }

// Entry p ends a list when it is negative (padding), or bad: at or beyond the source's
// filled blocks, or not above the entry before it. 2 p + bad then, or the largest int.
__device__ __forceinline__ int list_end(const int32_t *list, int p, int avail) {
    const int e = __ldg(list + p), before = p > 0 ? __ldg(list + p - 1) : -1;
    return e < 0 ? 2 * p : e >= avail || e <= before ? 2 * p + 1 : 0x7fffffff;
}

__device__ __forceinline__ int source_blocks(const CopyArgs &a, int job) {
    const int s = a.src_slot[job];
    return s >= 0 && s < a.src_batch ? filled(a.src_n, s, a.src_cap) : 0;
}

__global__ void __launch_bounds__(256) copy_check_kernel(CopyArgs a) {
    __shared__ int first;
    grid_dep_launch();
    const int job = blockIdx.y, p0 = blockIdx.x * kCheckPart;
    const int avail = source_blocks(a, job);
    const int32_t *list = a.keep + (size_t)job * a.cols;
    if (threadIdx.x == 0) first = 0x7fffffff;
    __syncthreads();
    int mine = 0x7fffffff;
#pragma unroll 4
    for (int k = 0; k < kCheckPart / 256; ++k) {
        const int p = p0 + k * 256 + threadIdx.x;
        if (p < a.cols) mine = min(mine, list_end(list, p, avail));
    }
    if (mine != 0x7fffffff) atomicMin(&first, mine);
    for (int t = threadIdx.x; t < kCheckPart / kTileRows; t += blockDim.x) {
        const int tile = p0 / kTileRows + t;
        if (tile < a.list_tiles) a.flags[(size_t)job * a.list_tiles + tile] = 0;
    }
    __syncthreads();
    if (threadIdx.x == 0) a.part_end[(size_t)job * a.parts + blockIdx.x] = first == 0x7fffffff ? -1 : first;
}

__global__ void __launch_bounds__(kPlanThreads) copy_plan_kernel(CopyArgs a) {
    __shared__ int s_tab[3 * kPlanSmemBatch];
    __shared__ long long scan_tmp[32];
    __shared__ long long round_total;
    grid_dep_wait();
    grid_dep_launch();
    if (a.plan_lists) {
        for (int i = threadIdx.x >> 5; i < a.jobs; i += kPlanThreads / 32) {
            const int avail = source_blocks(a, i), lane = threadIdx.x & 31;
            const int32_t *list = a.keep + (size_t)i * a.cols;
            int mine = 0x7fffffff;
#pragma unroll 4
            for (int p = lane; p < a.cols; p += 32) mine = min(mine, list_end(list, p, avail));
            mine = __reduce_min_sync(0xffffffffu, mine);
            if (lane == 0) a.part_end[i] = mine == 0x7fffffff ? -1 : mine;
        }
        for (int t = threadIdx.x; t < a.jobs * a.list_tiles; t += kPlanThreads) a.flags[t] = 0;
    }
    const int B = a.dst_batch;
    int *first = B <= kPlanSmemBatch ? s_tab : a.slot_tab;  // lowest job that writes a slot
    int *src_lo = first + B, *src_hi = src_lo + B;          // lowest and highest job that reads it
    auto seen = [](const int *p) { return *reinterpret_cast<const volatile int *>(p); };  // what atomics left
    for (int b = threadIdx.x; b < B; b += blockDim.x) {
        first[b] = 0x7fffffff;
        src_lo[b] = 0x7fffffff;
        src_hi[b] = -1;
    }
    __threadfence_block();
    __syncthreads();
    for (int i = threadIdx.x; i < a.jobs; i += blockDim.x) {
        const int s = a.src_slot[i], d = a.dst_slot[i];
        if (d >= 0 && d < B) atomicMin(first + d, i);
        if (a.same && s >= 0 && s < B) {
            atomicMin(src_lo + s, i);
            atomicMax(src_hi + s, i);
        }
    }
    __threadfence_block();
    __syncthreads();
    // counts and refusals (n_blocks is only read here; it is written below)
    for (int i = threadIdx.x; i < a.jobs; i += blockDim.x) {
        const int s = a.src_slot[i], d = a.dst_slot[i];
        int n = -1, bad = 0;
        if (d < 0 || d >= B || s >= a.src_batch || seen(first + d) != i) {
            bad = CSA_DEV_BAD_INDEX;
        } else if (a.same && (seen(src_lo + d) < i || seen(src_hi + d) > i) && !(s == d && !a.keep)) {
            bad = CSA_DEV_BAD_INDEX;  // another job reads what this one would overwrite
        } else {
            n = 0;
            if (s >= 0) {
                n = filled(a.src_n, s, a.src_cap);
                if (a.keep) {
                    n = a.cols;
                    for (int p = 0; p < a.parts; ++p) {
                        const int e = a.part_end[(size_t)i * a.parts + p];
                        if (e >= 0) {
                            n = e >> 1;
                            if (e & 1) bad = CSA_DEV_BAD_INDEX;
                            break;
                        }
                    }
                }
                if (a.max_blocks) n = min(n, max(a.max_blocks[i], 0));
            }
            if (n > a.dst_cap) {
                n = -1;
                bad |= CSA_DEV_CAPACITY;
            }
        }
        if (bad) flag(a.status, bad);
        JobRec r = {s, d, n, 0};
        a.rec[i] = r;
    }
    __threadfence_block();
    __syncthreads();
    long long carry = 0;
    for (int base = 0; base < a.jobs; base += blockDim.x) {
        const int i = base + threadIdx.x;
        long long tiles = 0;
        if (i < a.jobs) {
            const JobRec r = a.rec[i];
            // a job that follows one with the same source and count, within an aligned run of kFan, shares its tiles
            auto shares = [&](int k) {  // job k goes with job k - 1
                if (a.keep || k % kFan == 0 || k >= a.jobs) return false;
                const JobRec x = a.rec[k - 1], y = a.rec[k];
                return x.n > 0 && x.n == y.n && x.src == y.src && !(a.same && (x.src == x.dst || y.src == y.dst));
            };
            const bool moves = r.n > 0 && !(a.same && r.src == r.dst && !a.keep);
            if (moves && !shares(i)) {
                int f = 0;
                while (shares(i + f + 1)) ++f;
                a.rec[i].followers = f;
                tiles = (r.n + kTileRows - 1) / kTileRows;
            }
            if (r.n >= 0) a.dst_n[r.dst] = r.n;
        }
        const long long incl = block_inclusive_scan<long long>(tiles, scan_tmp);
        if (i < a.jobs) a.prefix[i + 1] = carry + incl;
        if (threadIdx.x == blockDim.x - 1) round_total = incl;
        __syncthreads();
        carry += round_total;
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        a.prefix[0] = 0;
        *a.ticket = 0;
    }
}

// ---- bytes between global and shared memory, by all threads of the block
__device__ __forceinline__ uint32_t unit_of(uintptr_t differing) {  // 16, 8, 4 or 1
    return (differing & 15) == 0 ? 16u : (differing & 7) == 0 ? 8u : (differing & 3) == 0 ? 4u : 1u;
}

__device__ __forceinline__ void copy_in_unit(uint32_t to, const uint8_t *from, uint32_t unit) {
    if (unit == 16) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    } else if (unit == 8) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
    } else if (unit == 4) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
    } else {
        const uint32_t v = *from;
        asm volatile("st.shared.u8 [%0], %1;" ::"r"(to), "r"(v) : "memory");
    }
}

// n bytes at `from` to shared address `to`
__device__ __forceinline__ void copy_in(uint32_t to, const uint8_t *from, uint32_t n) {
    const uint32_t unit = unit_of(reinterpret_cast<uintptr_t>(from) ^ to);
    const uint32_t head = min(n, (uint32_t)(0 - reinterpret_cast<uintptr_t>(from)) & (unit - 1));
    const uint32_t body = (n - head) / unit, tail = head + body * unit;
    if (threadIdx.x < head) copy_in_unit(to + threadIdx.x, from + threadIdx.x, 1);
    for (uint32_t k = threadIdx.x; k < body; k += kMoveThreads)
        copy_in_unit(to + head + k * unit, from + head + (size_t)k * unit, unit);
    if (tail + threadIdx.x < n) copy_in_unit(to + tail + threadIdx.x, from + tail + threadIdx.x, 1);
}

// n bytes of shared memory at `from` to `to`
__device__ __forceinline__ void copy_out(uint8_t *to, const uint8_t *from, uint32_t n) {
    const uint32_t unit = unit_of(reinterpret_cast<uintptr_t>(to) ^ smem_u32(from));
    const uint32_t head = min(n, (uint32_t)(0 - reinterpret_cast<uintptr_t>(to)) & (unit - 1));
    const uint32_t body = (n - head) / unit, tail = head + body * unit;
    if (threadIdx.x < head) to[threadIdx.x] = from[threadIdx.x];
    for (uint32_t k = threadIdx.x; k < body; k += kMoveThreads) {
        const uint32_t o = head + k * unit;
        if (unit == 16) *reinterpret_cast<uint4 *>(to + o) = *reinterpret_cast<const uint4 *>(from + o);
        else if (unit == 8) *reinterpret_cast<uint2 *>(to + o) = *reinterpret_cast<const uint2 *>(from + o);
        else if (unit == 4) *reinterpret_cast<uint32_t *>(to + o) = *reinterpret_cast<const uint32_t *>(from + o);
        else to[o] = from[o];
    }
    if (tail + threadIdx.x < n) to[tail + threadIdx.x] = from[tail + threadIdx.x];
}

// First position in the ascending list[0, n) whose entry is >= v, by one warp: 32 probes a step.
template <typename T>
__device__ __forceinline__ int lower_bound_warp(const T *list, int n, T v) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;  // the answer lies in [lo, hi]
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const int p = lo + lane * step;
        const bool below = p < hi && list[p] < v;
        const int k = __popc(__ballot_sync(0xffffffffu, below));  // probes below v: a prefix of the lanes
        if (k == 0) return lo;
        const int last = lo + (k - 1) * step;  // below v
        hi = min(hi, last + step);
        lo = last + 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kMoveThreads) cache_move_kernel(CopyArgs a) {
    extern __shared__ __align__(16) uint8_t buf[];
    __shared__ int s_idx[2][kTileRows];
    __shared__ long long s_ticket;
    __shared__ int s_dep[2];
    __shared__ int s_late;
    grid_dep_wait();
    const long long total = a.prefix[a.jobs];
    const int warp = threadIdx.x >> 5;
    struct Tile {
        int job, tile;
        JobRec r;
    };
    // Where tile t lies, and its list entries on their way to `idx`. The next tile's are found while the rows of this
    // one load: five dependent loads or more that every tile used to begin with (318 us for the 32 slots above).
    auto find = [&](long long t, int *idx) {
        Tile x = {};
        if (t < total) {
            x.job = lower_bound_warp(a.prefix + 1, a.jobs - 1, t + 1);  // prefix[job] <= t < prefix[job + 1]
            x.r = a.rec[x.job];
            x.tile = (int)(t - a.prefix[x.job]);
            const int k = x.tile * kTileRows + threadIdx.x;
            if (a.keep && threadIdx.x < kTileRows && k < x.r.n) idx[threadIdx.x] = __ldg(a.keep + (size_t)x.job * a.cols + k);
        }
        return x;
    };
    if (threadIdx.x == 0) s_ticket = (long long)atomicAdd(a.ticket, 1ull);
    __syncthreads();
    long long t = s_ticket, t_next;
    Tile now = find(t, s_idx[0]), next;
    for (int cur = 0; t < total; t = t_next, now = next, cur ^= 1) {
        const JobRec r = now.r;
        const int lo = now.job, tile = now.tile, j0 = tile * kTileRows, rows = min(kTileRows, r.n - j0);
        const int32_t *list = a.keep ? a.keep + (size_t)lo * a.cols : nullptr;
        const bool in_place = a.same && r.src == r.dst;
        const int *idx = s_idx[cur];
        __syncthreads();  // the indices are there; everyone has read s_ticket and left the buffers of the tile before
        if (threadIdx.x == 0) {
            s_ticket = (long long)atomicAdd(a.ticket, 1ull);
            s_late = 0;
        }
        const uint32_t buf_s = smem_u32(buf);
        // an in-place tile whose blocks stay where they are: ascending, so the two ends tell
        const bool still = in_place && idx[0] == j0 && idx[rows - 1] == j0 + rows - 1;
        uint32_t at[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q >= a.planes) break;
            const Plane pl = a.plane[q];
            // the tile sits in shared memory at its first destination's offset from a 16-byte boundary
            const size_t dst_at = ((size_t)r.dst * a.dst_cap + j0) * pl.row;
            at[q] = pl.at + (uint32_t)((reinterpret_cast<uintptr_t>(pl.dst) + dst_at) & 15);
            if (still) continue;
            const uint8_t *src = pl.src + (size_t)r.src * a.src_cap * pl.row;
            if (!list) {
                copy_in(buf_s + at[q], src + (size_t)j0 * pl.row, (uint32_t)rows * pl.row);
            } else {
                const uint32_t unit = unit_of(reinterpret_cast<uintptr_t>(src) | (buf_s + at[q]) | (uint32_t)pl.row);
                const uint32_t per = pl.row / unit, n = rows * per;
                if (unit == 16 && (per & (per - 1)) == 0) {  // as a rule: no division, four loads a turn
                    const int shift = __ffs(per) - 1;
#pragma unroll 4
                    for (uint32_t k = threadIdx.x; k < n; k += kMoveThreads) {
                        const uint32_t row = k >> shift, o = (k & (per - 1)) * 16;
                        copy_in_unit(buf_s + at[q] + k * 16, src + (size_t)idx[row] * pl.row + o, 16);
                    }
                } else {
                    for (uint32_t k = threadIdx.x; k < n; k += kMoveThreads) {
                        const uint32_t row = k / per, o = (k - row * per) * unit;
                        copy_in_unit(buf_s + at[q] + row * pl.row + o, src + (size_t)idx[row] * pl.row + o, unit);
                    }
                }
            }
        }
        if (in_place && !still && warp < 2) {  // positions of the list whose sources lie in [j0, j0 + rows)
            const int p = lower_bound_warp(list, min(r.n, j0 + rows), warp == 0 ? j0 : j0 + rows);
            if ((threadIdx.x & 31) == 0) s_dep[warp] = p;
        }
        __syncthreads();  // s_ticket
        t_next = s_ticket;
        next = find(t_next, s_idx[cur ^ 1]);
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        if (in_place) {
            int *fl = a.flags + (size_t)lo * a.list_tiles;
#ifdef CSA_TEST_LOST_ARRIVALS  // a test build in which the tiles that wait for a job's first one wait in vain
            if (threadIdx.x == 0 && tile != 0) {
#else
            if (threadIdx.x == 0) {
#endif
                __threadfence();
                asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(fl + tile), "r"(1) : "memory");
            }
            if (!still && s_dep[1] > s_dep[0]) {
                const int d0 = s_dep[0] / kTileRows, d1 = (s_dep[1] - 1) / kTileRows;
                for (int d = d0 + (int)threadIdx.x; d <= d1; d += kMoveThreads) {
                    const long long began = clock64();
                    int done = d == tile;
                    while (!done) {
                        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(done) : "l"(fl + d) : "memory");
                        if (!done && clock64() - began > kWaitCycles) {
                            s_late = 1;
                            break;
                        }
                    }
                }
            }
            __syncthreads();
            // Never written over blocks that were not read. The slot then ends before the first such tile (later ones
            // may be written), so that no old block counts as a kept one, with a status word or without.
            if (s_late) {
                if (threadIdx.x == 0) {
                    atomicMin(a.dst_n + r.dst, j0);
                    flag(a.status, CSA_DEV_TIMEOUT);
                }
                continue;
            }
        }
        if (!still) {
            for (int f = 0; f <= r.followers; ++f) {
                const int d = f == 0 ? r.dst : a.rec[lo + f].dst;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q >= a.planes) break;
                    const Plane pl = a.plane[q];
                    copy_out(pl.dst + ((size_t)d * a.dst_cap + j0) * pl.row, buf + at[q], (uint32_t)rows * pl.row);
                }
            }
        }
    }
}

struct Layout {
    size_t rec, prefix, ticket, slot_tab, part_end, flags, bytes;
    int parts, list_tiles;
};

Layout layout_of(int dst_batch, int jobs, int cols) {
    Layout l;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) & ~size_t(255);
        return at;
    };
    l.parts = (cols + kCheckPart - 1) / kCheckPart;
    l.list_tiles = (cols + kTileRows - 1) / kTileRows;
    l.rec = take(sizeof(JobRec) * (size_t)jobs);
    l.prefix = take(8 * ((size_t)jobs + 1));
    l.ticket = take(8);
    l.slot_tab = take(dst_batch > kPlanSmemBatch ? 12 * (size_t)dst_batch : 0);
    l.part_end = take(4 * (size_t)jobs * l.parts);
    l.flags = take(4 * (size_t)jobs * l.list_tiles);
    l.bytes = off;
    return l;
}

}  // namespace

size_t cache_copy_workspace_bytes(int dst_batch, int jobs, int cols) { return layout_of(dst_batch, jobs, cols).bytes; }

cudaError_t launch_cache_copy(const csa_cache &src, const csa_cache &dst, int jobs, const int32_t *src_slot,
                              const int32_t *dst_slot, const int32_t *keep, int cols, const int32_t *max_blocks,
                              void *workspace, int num_sms, cudaStream_t s) {
    const Layout l = layout_of(dst.batch, jobs, keep ? cols : 0);
    char *base = static_cast<char *>(workspace);
    CopyArgs a = {};
    int at = 0;
    auto plane = [&](const void *from, void *to, int row) {
        a.plane[a.planes++] = {static_cast<const uint8_t *>(from), static_cast<uint8_t *>(to), row, at};
        at += tile_bytes(row);
    };
    plane(src.fp4, dst.fp4, src.dim / 2);
    plane(src.scale, dst.scale, src.dim / (src.scale_fmt == CSA_SCALE_E4M3_16 ? 16 : 32));
    if (src.idx_key) {
        const int d = src.idx_dim;
        plane(src.idx_key, dst.idx_key,
              src.idx_dtype == CSA_IDX_BF16 ? 2 * d : src.idx_dtype == CSA_IDX_E4M3 ? d : d / 2);
        if (src.idx_dtype == CSA_IDX_MXFP4) plane(src.idx_key_scale, dst.idx_key_scale, d / 32);
    }
    a.src_batch = src.batch;
    a.src_cap = src.capacity;
    a.dst_batch = dst.batch;
    a.dst_cap = dst.capacity;
    a.same = src.fp4 == dst.fp4;
    a.src_n = src.n_blocks;
    a.dst_n = dst.n_blocks;
    a.status = dst.status;
    a.src_slot = src_slot;
    a.dst_slot = dst_slot;
    a.keep = keep;
    a.max_blocks = max_blocks;
    a.jobs = jobs;
    a.cols = cols;
    a.plan_lists = keep && cols <= kCheckPart && (long long)jobs * cols <= kPlanEntries;
    a.parts = l.parts;  // (1 where the plan kernel reads the lists: it writes no other part's end)
    a.list_tiles = l.list_tiles;
    a.rec = reinterpret_cast<JobRec *>(base + l.rec);
    a.prefix = reinterpret_cast<long long *>(base + l.prefix);
    a.ticket = reinterpret_cast<unsigned long long *>(base + l.ticket);
    a.slot_tab = reinterpret_cast<int *>(base + l.slot_tab);
    a.part_end = reinterpret_cast<int *>(base + l.part_end);
    a.flags = reinterpret_cast<int *>(base + l.flags);
    // One limit for every layout: it belongs to the kernel, and threads that set their own call's could lower it between
    // another's setting and its launch. Before the plan, which already writes n_blocks.
    cudaError_t err = cudaFuncSetAttribute(cache_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostTileBytes);
    if (err != cudaSuccess) return err;
    if (keep && !a.plan_lists) {
        copy_check_kernel<<<dim3(l.parts, jobs), 256, 0, s>>>(a);
        if ((err = cudaGetLastError()) != cudaSuccess) return err;
        if ((err = launch_pdl(copy_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a)) != cudaSuccess) return err;
    } else {
        copy_plan_kernel<<<1, kPlanThreads, 0, s>>>(a);
        if ((err = cudaGetLastError()) != cudaSuccess) return err;
    }
    // as many thread blocks as fit an SM's shared memory, up to its 2048 threads; no more than there can be tiles
    const long long most = (long long)jobs * (((long long)(keep ? min(cols, dst.capacity) : dst.capacity) + kTileRows - 1) / kTileRows);
    const long long grid = min(most, (long long)num_sms * max(1, min(8, 220 * 1024 / (at + 2048))));
    return launch_pdl(cache_move_kernel, dim3((unsigned)grid), dim3(kMoveThreads), (size_t)at, s, a);
}

}  // namespace csa
