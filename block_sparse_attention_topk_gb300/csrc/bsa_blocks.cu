// bsa_blocks.cu -- what becomes of a paged cache's blocks between steps:
// requests forked, reordered, grown and freed, and the blocks in use moved
// together.
//
// Both operators are a plan and its application.  The plan is integer work on
// tables of kilobytes to a few megabytes with a chain of dependent phases
// (counts before a scan, a scan before ids), so it is one cluster of 8 CTAs
// (or one CTA, where there is little to read)
// whose barrier separates the phases: no second launch for each, and no
// waiting on CTAs that may not be resident.  The application writes the table
// and copies whole blocks of every tensor, over the whole GPU.
//
// Measured: 20480 blocks of 4 heads of 128 in bf16 (5.4 GB), 5100 of them moved, 425 us, 0.94 of a copy's rate,
// with 32 KB a CTA in flight; 512 beams of 128 requests, about 155 unfinished blocks copied (262 KB each), 31 us, of
// which the plan is about 12 (five phases, each a chain of reads from L2); four beams 11 us, by one CTA (by the
// cluster 13), a small compaction 9 us (14).
//
// Order and ties: free blocks are taken from the lowest id on, in order of
// (row, block); counts are integer atomics, whose order does not show.
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include <algorithm>

#include "bsa_internal.h"
#include "bsa_overlap.h"
#include "bsa_tcgen05.cuh"

namespace bsa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kCluster = 8;
constexpr int kPlanThreads = 1024;
constexpr int64_t kOneCta = 16384;                          // entries and counts that one CTA plans
constexpr int kCopyThreads = 256;
constexpr int kUnroll = 8;                                   // 16-byte words of a thread in flight
constexpr int kChunk = kCopyThreads * kUnroll * 16;          // bytes of a tensor's block that a CTA copies at a time

// What the plan leaves in the workspace for the application, and its own counts.
struct Head {
    int32_t needed, available;        // fork: fresh blocks; compact: needed = blocks moved
    int32_t count[3][kCluster];
};

struct ForkParams {
    const int32_t* table;             // the old state as the kernels read it: the caller's, or its copy
    const int32_t* lens;
    const int32_t* table_in;          // the caller's, copied to table / lens first where they differ
    const int32_t* lens_in;
    int32_t* snap_table;
    int32_t* snap_lens;
    const int32_t* refs_in;
    const int32_t* parent;
    const int32_t* new_tokens;        // or null
    int32_t* table_out;
    int32_t* lens_out;
    int32_t* refs_out;
    int64_t rows_in, rows_out, max_blocks, num_blocks;
    Head* head;
    int32_t* first;                   // [rows_in] lowest new row of each old one
    struct RowPlan* rows;             // [rows_out]
    int32_t* fresh;                   // fresh block ids in order
    uint32_t* status;
    int32_t ranks;                    // CTAs of the plan: 1 or kCluster
};

// What the application needs of a row, in one read.
struct alignas(32) RowPlan {
    int32_t parent, shared, blocks;   // shared: the parent's blocks that are this row's too, its first
    int32_t offset;                   // its first fresh block's place in `fresh`
    int32_t copied;                   // the unfinished block to copy into that, or -1
    int32_t pad[3];
};

struct CompactParams {
    const int32_t* table;
    const int32_t* lens;
    const int32_t* refs_in;
    int32_t* table_out;
    int32_t* refs_out;
    int32_t* new_ids;
    int64_t rows, max_blocks, num_blocks;
    Head* head;
    int32_t *src, *dst, *src_refs;
    uint32_t* status;
    int32_t ranks;                    // CTAs of the plan: 1 or kCluster
};

// What a block's id stands for, as a launch's argument.
template <int MAX>
struct Tensors {
    uint8_t* p[MAX];
    int64_t bytes[MAX];                                      // of a block
    int32_t chunks[MAX + 1];                                 // chunks of a block before each tensor's
    int32_t n;
};
constexpr int kFewTensors = 16;      // 10 KB of arguments take longer to launch than the 350 bytes of these
using AllTensors = Tensors<BSA_MAX_BLOCK_TENSORS>;

__device__ __forceinline__ int64_t blocks_of(int64_t tokens) { return (tokens + kPageSize - 1) / kPageSize; }

// Phases of the plan: global memory written before is read after (from L2: __ldcg).
__device__ __forceinline__ void phase(int ranks) {
    if (ranks == 1) {
        __syncthreads();
        return;
    }
    __threadfence();
    cluster_sync();
}

// A length within the table.
__device__ __forceinline__ int64_t checked_len(int64_t n, int64_t max_blocks, uint32_t* status) {
    const int64_t top = max_blocks * kPageSize, m = n < 0 ? 0 : n > top ? top : n;
    report_status(status, m != n, BSA_STATUS_BAD_CONTEXT);
    return m;
}

// Inclusive sum over the CTA's 1024 threads, and the total.  `warps`: 32 words.
__device__ __forceinline__ int cta_scan(int x, int* warps, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = warps[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, w, o);
            if (lane >= o) w += y;
        }
        warps[lane] = w;
    }
    __syncthreads();
    *total = warps[31];
    return x + (warp > 0 ? warps[warp - 1] : 0);
}

struct Row {
    int64_t base, len;     // the parent's tokens, and the row's
    int32_t parent;        // or -1
};
__device__ __forceinline__ Row new_row(const ForkParams& P, const int32_t* lens, int64_t r, uint32_t* status) {
    Row w;
    const int32_t p = __ldg(P.parent + r);
    w.parent = p < 0 || p >= P.rows_in ? -1 : p;
    report_status(status, w.parent != p && p != -1, BSA_STATUS_BAD_CONTEXT);
    w.base = w.parent < 0 ? 0 : checked_len(__ldcg(lens + w.parent), P.max_blocks, nullptr);
    const int64_t more = P.new_tokens == nullptr ? 0 : __ldg(P.new_tokens + r);
    report_status(status, more < 0, BSA_STATUS_BAD_CONTEXT);
    w.len = checked_len(w.base + (more < 0 ? 0 : more), P.max_blocks, status);
    return w;
}

constexpr int kRowsKept = 1024;       // rows whose parents and lengths a CTA of the plan keeps

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkParams P) {
    __shared__ int warps[32];
    __shared__ Row kept[kRowsKept];
    const int tid = threadIdx.x, rank = blockIdx.x, all = rank * kPlanThreads + tid, everyone = P.ranks * kPlanThreads;
    const int lane = tid & 31, gwarp = all >> 5;
    asm volatile("griddepcontrol.launch_dependents;");
    // ---- the old state, where the new one takes its place; counts to start from
    if (P.refs_out != P.refs_in)
        for (int64_t i = all; i < P.num_blocks; i += everyone) P.refs_out[i] = __ldg(P.refs_in + i);
    if (P.snap_table != nullptr)
        for (int64_t i = all; i < P.rows_in * P.max_blocks; i += everyone) P.snap_table[i] = P.table_in[i];
    if (P.snap_lens != nullptr)
        for (int64_t i = all; i < P.rows_in; i += everyone) P.snap_lens[i] = P.lens_in[i];
    for (int64_t i = all; i < P.rows_in; i += everyone) P.first[i] = INT_MAX;
    // a row is a chain of reads (its parent, that one's length): once for all phases where they fit.  From the
    // caller's lengths: they are not written before the third phase
    const bool keep = P.rows_out <= kRowsKept;
    if (keep && tid < P.rows_out) kept[tid] = new_row(P, P.lens_in, tid, rank == 0 ? P.status : nullptr);
    auto row = [&](int64_t r) { return keep ? kept[r] : new_row(P, P.lens, r, nullptr); };
    phase(P.ranks);
    // ---- references of whole blocks: a warp per old and per new row
    for (int64_t i = all; i < P.rows_out; i += everyone) {
        const Row w = keep ? kept[i] : new_row(P, P.lens, i, P.status);
        if (w.parent >= 0) atomicMin(P.first + w.parent, (int)i);
    }
    for (int64_t r = gwarp; r < P.rows_in; r += everyone / 32) {
        const int64_t len = checked_len(__ldcg(P.lens + r), P.max_blocks, lane == 0 ? P.status : nullptr);
        const bool stays = r < P.rows_out && __ldg(P.parent + r) == r;      // its whole blocks stay its own
        for (int64_t j = (stays ? len / kPageSize : 0) + lane; j < blocks_of(len); j += 32) {
            const int32_t b = __ldcg(P.table + r * P.max_blocks + j);
            const bool good = b >= 0 && b < P.num_blocks;
            report_status(P.status, !good, BSA_STATUS_BAD_BLOCK_ID);
            if (good) atomicSub(P.refs_out + b, 1);
        }
    }
    for (int64_t r = gwarp; r < P.rows_out; r += everyone / 32) {
        const Row w = row(r);
        if (w.parent < 0 || w.parent == r) continue;
        for (int64_t j = lane; j < w.base / kPageSize; j += 32) {
            const int32_t b = __ldcg(P.table + w.parent * P.max_blocks + j);
            if (b >= 0 && b < P.num_blocks) atomicAdd(P.refs_out + b, 1);
        }
    }
    phase(P.ranks);
    // ---- unfinished blocks go to the first child; fresh blocks of each row, in order
    if (rank == 0) {
        int before = 0;
        for (int64_t r0 = 0; r0 < P.rows_out; r0 += kPlanThreads) {
            const int64_t r = r0 + tid;
            int need = 0, copy = -1;
            Row w{0, 0, -1};
            if (r < P.rows_out) {
                w = row(r);
                need = (int)(blocks_of(w.len) - blocks_of(w.base));
                if (w.base % kPageSize != 0) {
                    const int32_t b = __ldcg(P.table + w.parent * P.max_blocks + w.base / kPageSize);
                    if (__ldcg(P.first + w.parent) != (int)r) {
                        ++need;
                        copy = b >= 0 && b < P.num_blocks ? b : INT_MAX;       // INT_MAX: a block without contents
                    } else if (b >= 0 && b < P.num_blocks) {
                        atomicAdd(P.refs_out + b, 1);
                    }
                }
                P.lens_out[r] = (int32_t)w.len;
            }
            int total;
            const int upto = before + cta_scan(need, warps, &total);
            if (r < P.rows_out) {
                RowPlan p;
                p.parent = w.parent;
                p.shared = (int32_t)blocks_of(w.base) - (copy >= 0);
                p.blocks = (int32_t)blocks_of(w.len);
                p.offset = upto - need;
                p.copied = copy;
                P.rows[r] = p;
            }
            before += total;
        }
        if (tid == 0) P.head->needed = before;
    }
    phase(P.ranks);
    // ---- the lowest free blocks: counted per CTA's share, then listed
    const int64_t lo = P.num_blocks * rank / P.ranks, hi = P.num_blocks * (rank + 1) / P.ranks;
    int mine = 0;
    for (int64_t i = lo + tid; i < hi; i += kPlanThreads) mine += __ldcg(P.refs_out + i) <= 0;
    int total;
    cta_scan(mine, warps, &total);
    if (tid == 0) P.head->count[0][rank] = total;
    phase(P.ranks);
    int before = 0, available = 0;
    for (int i = 0; i < P.ranks; ++i) {
        const int n = __ldcg(&P.head->count[0][i]);
        if (i < rank) before += n;
        available += n;
    }
    const int needed = __ldcg(&P.head->needed);
    if (rank == 0 && tid == 0) {
        P.head->available = available;
        report_status(P.status, needed > available, BSA_STATUS_NO_BLOCK);
    }
    for (int64_t i0 = lo; i0 < hi && before < needed; i0 += kPlanThreads) {
        const int64_t i = i0 + tid;
        const int free = i < hi && __ldcg(P.refs_out + i) <= 0;
        const int at = before + cta_scan(free, warps, &total) - free;
        if (free && at < needed) {
            P.fresh[at] = (int32_t)i;
            P.refs_out[i] = 1;
        }
        before += total;
    }
}

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactParams P) {
    __shared__ int warps[32];
    const int tid = threadIdx.x, rank = blockIdx.x, everyone = P.ranks * kPlanThreads;
    asm volatile("griddepcontrol.launch_dependents;");
    const int64_t lo = P.num_blocks * rank / P.ranks, hi = P.num_blocks * (rank + 1) / P.ranks;
    int mine = 0, total;
    for (int64_t i = lo + tid; i < hi; i += kPlanThreads) mine += __ldcg(P.refs_in + i) > 0;
    cta_scan(mine, warps, &total);
    if (tid == 0) P.head->count[0][rank] = total;
    phase(P.ranks);
    int live = 0;
    for (int i = 0; i < P.ranks; ++i) live += __ldcg(&P.head->count[0][i]);
    // ---- blocks to move and holes to fill, counted per share
    int moving = 0, holes = 0;
    for (int64_t i = lo + tid; i < hi; i += kPlanThreads) {
        const bool used = __ldcg(P.refs_in + i) > 0;
        moving += used && i >= live;
        holes += !used && i < live;
    }
    cta_scan(moving, warps, &total);
    if (tid == 0) P.head->count[1][rank] = total;
    cta_scan(holes, warps, &total);
    if (tid == 0) P.head->count[2][rank] = total;
    phase(P.ranks);
    int moved_before = 0, holes_before = 0, moves = 0;
    for (int i = 0; i < P.ranks; ++i) {
        const int m = __ldcg(&P.head->count[1][i]), h = __ldcg(&P.head->count[2][i]);
        if (i < rank) {
            moved_before += m;
            holes_before += h;
        }
        moves += m;
    }
    if (rank == 0 && tid == 0) P.head->needed = moves;
    for (int64_t i0 = lo; i0 < hi; i0 += kPlanThreads) {
        const int64_t i = i0 + tid;
        const int refs = i < hi ? __ldcg(P.refs_in + i) : 0;
        const int move = i < hi && refs > 0 && i >= live, hole = i < hi && refs <= 0 && i < live;
        int m_total, h_total;
        const int m_at = moved_before + cta_scan(move, warps, &m_total) - move;
        const int h_at = holes_before + cta_scan(hole, warps, &h_total) - hole;
        if (move) {
            P.src[m_at] = (int32_t)i;
            P.src_refs[m_at] = refs;
        }
        if (hole) P.dst[h_at] = (int32_t)i;
        if (i < hi) {
            P.new_ids[i] = refs > 0 && i < live ? (int32_t)i : -1;
            P.refs_out[i] = refs > 0 && i < live ? refs : 0;
        }
        moved_before += m_total;
        holes_before += h_total;
    }
    phase(P.ranks);
    for (int64_t k = rank * kPlanThreads + tid; k < moves; k += everyone) {
        const int32_t from = __ldcg(P.src + k), to = __ldcg(P.dst + k);
        P.new_ids[from] = to;
        P.refs_out[to] = __ldcg(P.src_refs + k);
    }
}

// Chunk `c` of a block's tensors from block src to block dst.
template <int MAX>
__device__ __forceinline__ void copy_chunk(const Tensors<MAX>& X, int c, int64_t src, int64_t dst) {
    int t = 0;
    while (c >= X.chunks[t + 1]) ++t;
    const int64_t at = (int64_t)(c - X.chunks[t]) * kChunk, words = (X.bytes[t] - at) / 16;
    const uint4* from = reinterpret_cast<const uint4*>(X.p[t] + src * X.bytes[t] + at);
    uint4* to = reinterpret_cast<uint4*>(X.p[t] + dst * X.bytes[t] + at);
    uint4 v[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
        if (k * kCopyThreads + (int)threadIdx.x < words) v[k] = __ldcs(from + k * kCopyThreads + threadIdx.x);
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
        if (k * kCopyThreads + (int)threadIdx.x < words) __stcs(to + k * kCopyThreads + threadIdx.x, v[k]);
}

template <int MAX>
__global__ void __launch_bounds__(kCopyThreads) fork_apply_kernel(const ForkParams P, const __grid_constant__ Tensors<MAX> X) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int available = __ldcg(&P.head->available);
    const int chunks = X.chunks[X.n];
    for (int64_t i = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; i < P.rows_out * P.max_blocks; i += (int64_t)gridDim.x * kCopyThreads) {
        const int64_t r = i / P.max_blocks, j = i - r * P.max_blocks;
        const RowPlan w = P.rows[r];
        int32_t b = -1;
        if (j < w.shared) {
            // the plan reads the full blocks of requests that change rows alone
            b = __ldcg(P.table + w.parent * P.max_blocks + j);
            report_status(P.status, b < 0 || b >= P.num_blocks, BSA_STATUS_BAD_BLOCK_ID);
        } else if (j < w.blocks) {
            const int64_t k = w.offset + (j - w.shared);
            if (k < available) b = __ldcg(P.fresh + k);
        }
        P.table_out[i] = b;
    }
    for (int64_t i = blockIdx.x; i < P.rows_out * chunks; i += gridDim.x) {
        const int64_t r = i / chunks;
        const RowPlan w = P.rows[r];
        if (w.copied < 0 || w.copied == INT_MAX || w.offset >= available) continue;
        copy_chunk(X, (int)(i - r * chunks), w.copied, __ldcg(P.fresh + w.offset));
    }
}

template <int MAX>
__global__ void __launch_bounds__(kCopyThreads) compact_apply_kernel(const CompactParams P, const __grid_constant__ Tensors<MAX> X) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t moves = __ldcg(&P.head->needed);
    const int chunks = X.chunks[X.n];
    // row by row, as a table of no columns has rows too
    for (int64_t r = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; r < P.rows; r += (int64_t)gridDim.x * kCopyThreads)
        checked_len(__ldg(P.lens + r), P.max_blocks, P.status);
    for (int64_t i = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; i < P.rows * P.max_blocks; i += (int64_t)gridDim.x * kCopyThreads) {
        const int64_t r = i / P.max_blocks, j = i - r * P.max_blocks;
        const int64_t len = checked_len(__ldg(P.lens + r), P.max_blocks, nullptr);
        int32_t b = -1;
        if (j < blocks_of(len)) {
            const int32_t old = P.table[i];
            if (old >= 0 && old < P.num_blocks) b = __ldcg(P.new_ids + old);
            report_status(P.status, b < 0, BSA_STATUS_BAD_BLOCK_ID);
        }
        P.table_out[i] = b;
    }
    for (int64_t i = blockIdx.x; i < moves * chunks; i += gridDim.x) {
        const int64_t k = i / chunks;
        copy_chunk(X, (int)(i - k * chunks), __ldcg(P.src + k), __ldcg(P.dst + k));
    }
}

// ---- host ------------------------------------------------------------------

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Places of the workspace, in order; a null base counts.
struct Carve {
    uint8_t* base;
    size_t used = 0;
    template <typename T>
    T* take(int64_t n) {
        T* p = reinterpret_cast<T*>(base + used);
        used += up256((size_t)n * sizeof(T));
        return base == nullptr ? nullptr : p;
    }
};

size_t carve_fork(uint8_t* base, ForkParams* P, bool in_place) {
    Carve c{base};
    P->head = c.take<Head>(1);
    P->first = c.take<int32_t>(P->rows_in);
    P->rows = c.take<RowPlan>(P->rows_out);
    // each row needs max_blocks fresh blocks at most
    const int64_t all = P->rows_out * P->max_blocks;
    P->fresh = c.take<int32_t>(all < P->num_blocks ? all : P->num_blocks);
    int32_t* table = c.take<int32_t>(P->rows_in * P->max_blocks);
    int32_t* lens = c.take<int32_t>(P->rows_in);
    P->snap_table = in_place ? table : nullptr;
    P->snap_lens = in_place ? lens : nullptr;
    return c.used;
}

size_t carve_compact(uint8_t* base, CompactParams* P) {
    Carve c{base};
    P->head = c.take<Head>(1);
    P->src = c.take<int32_t>(P->num_blocks);
    P->dst = c.take<int32_t>(P->num_blocks);
    P->src_refs = c.take<int32_t>(P->num_blocks);
    return c.used;
}

bool blocks_sizes_ok(int64_t rows_in, int64_t rows_out, int64_t max_blocks, int64_t num_blocks) {
    const int64_t top = 1ll << 24;
    return rows_in >= 0 && rows_in <= top && rows_out >= 0 && rows_out <= top && max_blocks >= 0 && max_blocks < top &&
           num_blocks >= 0 && num_blocks <= BSA_MAX_PHYS_BLOCK && rows_in * max_blocks <= INT32_MAX && rows_out * max_blocks <= INT32_MAX;
}

int take_tensors(const bsa_block_tensor_t* t, int32_t n, AllTensors* X) {
    if (n < 0 || n > BSA_MAX_BLOCK_TENSORS) return BSA_ERR_SHAPE;
    if (n > 0 && t == nullptr) return BSA_ERR_NULL;
    X->n = n;
    X->chunks[0] = 0;
    for (int i = 0; i < n; ++i) {
        if (t[i].bytes_per_block < 0 || t[i].bytes_per_block > (1ll << 40)) return BSA_ERR_SHAPE;
        if (t[i].data == nullptr && t[i].bytes_per_block > 0) return BSA_ERR_NULL;
        if (t[i].bytes_per_block % 16 != 0 || (reinterpret_cast<uintptr_t>(t[i].data) & 15) != 0) return BSA_ERR_ALIGN;
        X->p[i] = static_cast<uint8_t*>(t[i].data);
        X->bytes[i] = t[i].bytes_per_block;
        const int64_t chunks = X->chunks[i] + (t[i].bytes_per_block + kChunk - 1) / kChunk;
        if (chunks > INT32_MAX / 2) return BSA_ERR_SHAPE;
        X->chunks[i + 1] = (int32_t)chunks;
    }
    return BSA_OK;
}

template <typename Params>
cudaError_t launch_pair(void (*plan)(const Params), void (*apply_few)(const Params, const Tensors<kFewTensors>),
                        void (*apply_all)(const Params, const AllTensors), const Params& P, const AllTensors& X, int64_t want,
                        cudaStream_t st) {
    cudaLaunchConfig_t one{};
    one.gridDim = dim3((unsigned)P.ranks);
    one.blockDim = dim3(kPlanThreads);
    one.stream = st;
    cudaLaunchAttribute cluster{};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = (unsigned)P.ranks;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    one.attrs = &cluster;
    one.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&one, plan, P);
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)device_sm_count() * 8;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(want < 1 ? 1 : want < most ? want : most));
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (X.n > kFewTensors) return cudaLaunchKernelEx(&cfg, apply_all, P, X);
    Tensors<kFewTensors> few{};
    for (int t = 0; t < X.n; ++t) {
        few.p[t] = X.p[t];
        few.bytes[t] = X.bytes[t];
        few.chunks[t + 1] = X.chunks[t + 1];
    }
    few.n = X.n;
    return cudaLaunchKernelEx(&cfg, apply_few, P, few);
}

Rows ints(const void* p, int64_t n) { return whole_rows(p, n * 4); }

// Nothing shares memory with the workspace.
bool apart_from(const Rows& scratch, const Rows* out, const Rows* in, int n_out, int n_in, const AllTensors& X, int64_t num_blocks) {
    for (int i = 0; i < n_out; ++i)
        if (rows_overlap(scratch, out[i])) return false;
    for (int j = 0; j < n_in; ++j)
        if (rows_overlap(scratch, in[j])) return false;
    for (int t = 0; t < X.n; ++t)
        if (rows_overlap(scratch, whole_rows(X.p[t], X.bytes[t] * num_blocks))) return false;
    return true;
}

// No output shares memory with an input (unless it is that input), another output or
// a tensor, and no tensor with another.
bool apart(const Rows* out, const Rows* in, int n_out, int n_in, const AllTensors& X, int64_t num_blocks) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j) {
            const bool itself = i == j && out[i].p == in[j].p;      // out i in the place of in i
            if (!itself && rows_overlap(out[i], in[j])) return false;
        }
        for (int j = i + 1; j < n_out; ++j)
            if (rows_overlap(out[i], out[j])) return false;
    }
    for (int t = 0; t < X.n; ++t) {
        const Rows x = whole_rows(X.p[t], X.bytes[t] * num_blocks);
        for (int i = 0; i < n_out; ++i)
            if (rows_overlap(x, out[i])) return false;
        for (int j = 0; j < n_in; ++j)
            if (rows_overlap(x, in[j])) return false;
    }
    int order[BSA_MAX_BLOCK_TENSORS], n = 0;
    for (int t = 0; t < X.n; ++t)
        if (X.bytes[t] > 0 && num_blocks > 0) order[n++] = t;
    std::sort(order, order + n, [&](int a, int b) { return X.p[a] < X.p[b]; });
    for (int i = 1; i < n; ++i)
        if (X.p[order[i]] - X.p[order[i - 1]] < X.bytes[order[i - 1]] * num_blocks) return false;
    return true;
}

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" size_t bsa_fork_workspace_bytes(int64_t rows_in, int64_t rows_out, int64_t max_blocks, int64_t num_blocks) {
    if (!blocks_sizes_ok(rows_in, rows_out, max_blocks, num_blocks)) return 0;
    ForkParams P{};
    P.rows_in = rows_in;
    P.rows_out = rows_out;
    P.max_blocks = max_blocks;
    P.num_blocks = num_blocks;
    return carve_fork(nullptr, &P, true);
}

extern "C" size_t bsa_compact_workspace_bytes(int64_t num_blocks) {
    if (!blocks_sizes_ok(0, 0, 0, num_blocks)) return 0;
    CompactParams P{};
    P.num_blocks = num_blocks;
    return carve_compact(nullptr, &P);
}

extern "C" int bsa_fork_requests(const bsa_block_tensor_t* tensors, int32_t num_tensors, const int32_t* block_table,
                                 const int32_t* seq_lens, const int32_t* block_refs, int64_t num_reqs, int64_t max_blocks,
                                 int64_t num_blocks, const int32_t* parent, const int32_t* new_tokens, int64_t num_out,
                                 int32_t* table_out, int32_t* lens_out, int32_t* refs_out, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    if (!blocks_sizes_ok(num_reqs, num_out, max_blocks, num_blocks)) return BSA_ERR_SHAPE;
    AllTensors X{};
    const int rc = take_tensors(tensors, num_tensors, &X);
    if (rc != BSA_OK) return rc;
    const int64_t in = num_reqs * max_blocks, out = num_out * max_blocks;
    if ((num_reqs > 0 && seq_lens == nullptr) || (in > 0 && block_table == nullptr) || (num_out > 0 && (parent == nullptr || lens_out == nullptr)) ||
        (out > 0 && table_out == nullptr) || (num_blocks > 0 && (block_refs == nullptr || refs_out == nullptr)))
        return BSA_ERR_NULL;
    if ((table_out == block_table && out != in) || (lens_out == seq_lens && num_out != num_reqs)) return BSA_ERR_SHAPE;
    const Rows outs[3] = {ints(table_out, out), ints(lens_out, num_out), ints(refs_out, num_blocks)};
    const Rows ins[5] = {ints(block_table, in), ints(seq_lens, num_reqs), ints(block_refs, num_blocks), ints(parent, num_out),
                         ints(new_tokens, new_tokens != nullptr ? num_out : 0)};
    if (!apart(outs, ins, 3, 5, X, num_blocks)) return BSA_ERR_SHAPE;
    ForkParams P{};
    P.rows_in = num_reqs;
    P.rows_out = num_out;
    P.max_blocks = max_blocks;
    P.num_blocks = num_blocks;
    const bool in_place = (in > 0 && table_out == block_table) || (num_reqs > 0 && lens_out == seq_lens);
    const size_t need = carve_fork(static_cast<uint8_t*>(workspace), &P, in_place);
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 || workspace_bytes < need) return BSA_ERR_WORKSPACE;
    if (!apart_from(whole_rows(workspace, (int64_t)need), outs, ins, 3, 5, X, num_blocks)) return BSA_ERR_SHAPE;
    P.table_in = block_table;
    P.lens_in = seq_lens;
    P.table = in_place ? P.snap_table : block_table;
    P.lens = in_place ? P.snap_lens : seq_lens;
    P.refs_in = block_refs;
    P.parent = parent;
    P.new_tokens = new_tokens;
    P.table_out = table_out;
    P.lens_out = lens_out;
    P.refs_out = refs_out;
    P.status = current_status_word();
    P.ranks = in + out + num_blocks <= kOneCta ? 1 : kCluster;
    const int64_t work = num_out * X.chunks[X.n], entries = (out + kCopyThreads - 1) / kCopyThreads;
    const cudaError_t e = launch_pair<ForkParams>(fork_plan_kernel, fork_apply_kernel<kFewTensors>, fork_apply_kernel<BSA_MAX_BLOCK_TENSORS>, P, X,
                                                   work > entries ? work : entries, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BSA_OK : (int)e;
}

extern "C" int bsa_compact_blocks(const bsa_block_tensor_t* tensors, int32_t num_tensors, const int32_t* block_table,
                                  const int32_t* seq_lens, const int32_t* block_refs, int64_t num_reqs, int64_t max_blocks,
                                  int64_t num_blocks, int32_t* table_out, int32_t* refs_out, int32_t* new_ids, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    if (!blocks_sizes_ok(num_reqs, num_reqs, max_blocks, num_blocks)) return BSA_ERR_SHAPE;
    AllTensors X{};
    const int rc = take_tensors(tensors, num_tensors, &X);
    if (rc != BSA_OK) return rc;
    const int64_t entries = num_reqs * max_blocks;
    if ((num_reqs > 0 && seq_lens == nullptr) || (entries > 0 && (block_table == nullptr || table_out == nullptr)) ||
        (num_blocks > 0 && (block_refs == nullptr || refs_out == nullptr || new_ids == nullptr)))
        return BSA_ERR_NULL;
    const Rows outs[3] = {ints(table_out, entries), ints(refs_out, num_blocks), ints(new_ids, num_blocks)};
    const Rows ins[3] = {ints(block_table, entries), ints(block_refs, num_blocks), ints(seq_lens, num_reqs)};
    if (new_ids != nullptr && static_cast<const int32_t*>(new_ids) == seq_lens) return BSA_ERR_SHAPE;
    if (!apart(outs, ins, 3, 3, X, num_blocks)) return BSA_ERR_SHAPE;
    CompactParams P{};
    P.rows = num_reqs;
    P.max_blocks = max_blocks;
    P.num_blocks = num_blocks;
    const size_t need = carve_compact(static_cast<uint8_t*>(workspace), &P);
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 || workspace_bytes < need) return BSA_ERR_WORKSPACE;
    if (!apart_from(whole_rows(workspace, (int64_t)need), outs, ins, 3, 3, X, num_blocks)) return BSA_ERR_SHAPE;
    P.table = block_table;
    P.lens = seq_lens;
    P.refs_in = block_refs;
    P.table_out = table_out;
    P.refs_out = refs_out;
    P.new_ids = new_ids;
    P.status = current_status_word();
    P.ranks = num_blocks <= kOneCta ? 1 : kCluster;
    // how many blocks move is known on the device alone: a full grid where many could
    const int64_t work = num_blocks * X.chunks[X.n], tables = (entries + kCopyThreads - 1) / kCopyThreads;
    const cudaError_t e = launch_pair<CompactParams>(compact_plan_kernel, compact_apply_kernel<kFewTensors>, compact_apply_kernel<BSA_MAX_BLOCK_TENSORS>, P, X,
                                                   work > tables ? work : tables, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BSA_OK : (int)e;
}
