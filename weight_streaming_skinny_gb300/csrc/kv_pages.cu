// Whose pages of the paged cache are: free, fork, reserve, compact (dl_kv_free, dl_kv_fork,
// dl_kv_reserve, dl_kv_compact).
#include "dl_device.cuh"
#include "dl_host.h"
#include "rows.cuh"

namespace dl {

// The state that all of them change, on the device: how many rows' tables name each page, the
// tables, the rows' lengths.  Results do not depend on timing: pages are taken from the lowest free
// number on, list items are served in their order, and counts change by atomic additions.
struct PageState {
    int *refs, *table, *lens;
    int num_pages, page_size, rows, cols;
};

// A row's length as its table can hold it.
__device__ __forceinline__ int row_len(const PageState& s, int row) {
    const long long room = (long long)s.cols * s.page_size;
    const int n = max(s.lens[row], 0);
    return (long long)n > room ? (int)room : n;
}
__device__ __forceinline__ int pages_for(const PageState& s, int len) {
    return (int)(((long long)len + s.page_size - 1) / s.page_size);
}
__device__ __forceinline__ bool in_pool(const PageState& s, int page) { return page >= 0 && page < s.num_pages; }

// What a listed item asks for and gets; in the workspace.
struct Plan {
    int row, from;         // the row that changes; fork: the row that it is a copy of
    int len, need, first;  // its length before (-1: refused), pages asked for, those asked for before it
    int src, dst;          // fork: the begun page and its copy (-1: nothing to copy)
    int tail;              // fork: tokens in the begun page; reserve: tokens asked for
};

constexpr int kPlanThreads = 1024;
constexpr int kMaxRows = 16384;          // `first` of the planning kernels fits shared memory

// Which of 16 pages from p on are free.
__device__ __forceinline__ unsigned free_mask(const PageState& s, int p) {
    unsigned m = 0;
    if (!((uintptr_t)s.refs & 15) && p + 16 <= s.num_pages) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint4 v = ldg128(s.refs + p + 4 * k);
            m |= ((int)v.x <= 0 ? 1u : 0u) << (4 * k) | ((int)v.y <= 0 ? 2u : 0u) << (4 * k) |
                 ((int)v.z <= 0 ? 4u : 0u) << (4 * k) | ((int)v.w <= 0 ? 8u : 0u) << (4 * k);
        }
    } else {
        for (int k = 0; k < 16; ++k)
            if (p + k < s.num_pages && s.refs[p + k] <= 0) m |= 1u << k;
    }
    return m;
}

// The first `want` free pages, lowest first, into list; returns how many there are (at most want).
// A thread looks at 16 pages a round; the first round's is done (`is_free`).
__device__ int free_pages(const PageState& s, int want, unsigned is_free, int* list, Scan& scan) {
    int found = 0;
    for (int p0 = 0; p0 < s.num_pages && found < want; p0 += 16 * kPlanThreads) {
        const int p = p0 + 16 * threadIdx.x;
        if (p0) is_free = free_mask(s, p);
        int total;
        const int n = __popc(is_free);
        int at = found + scan(n, total) - n;
        for (; is_free && at < want; ++at) {
            list[at] = p + __ffs(is_free) - 1;
            is_free &= is_free - 1;
        }
        found += total;
    }
    __syncthreads();
    return min(found, want);
}

// Give the listed rows' pages back: a CTA a row.  A row listed twice is given back once.
__global__ void __launch_bounds__(128) free_rows_kernel(PageState s, const int* rows) {
    __shared__ int pages;
    griddep_wait();
    griddep_launch_dependents();
    const int row = rows[blockIdx.x];
    if (row < 0 || row >= s.rows) return;
    if (threadIdx.x == 0) {
        const long long n = max(atomicExch(&s.lens[row], 0), 0);
        pages = (int)min((n + s.page_size - 1) / s.page_size, (long long)s.cols);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < pages; i += blockDim.x) {
        const int page = s.table[(size_t)row * s.cols + i];
        // a count that is used up stays where it is: who finds it so takes the step back
        if (in_pool(s, page) && atomicAdd(&s.refs[page], -1) <= 0) atomicAdd(&s.refs[page], 1);
    }
}

struct ListParams {
    PageState s;
    const int *a, *b;      // fork: parents and children; reserve: rows and tokens
    int* done;
    int n;
    Plan* plan;
    int* list;             // free pages
};

// Which listed items are served, with which pages; reserve is done by this.  One CTA: it is bound by its
// barriers' and loads' latency (5 to 6 us alone for 160 rows and 3000 pages), and lists are short.
template <bool FORK>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ ListParams p) {
    extern __shared__ int first[];       // of each row, the first item that changes it
    __shared__ int warp_sum[2][32];
    Scan scan{warp_sum};
    const PageState& s = p.s;
    const int tid = threadIdx.x;
    griddep_wait();
    griddep_launch_dependents();
    const unsigned is_free = free_mask(s, 16 * tid);     // (its loads overlap what follows)
    for (int i = tid; i < s.rows; i += kPlanThreads) first[i] = 0x7fffffff;
    __syncthreads();
    for (int i = tid; i < p.n; i += kPlanThreads) {
        const int row = FORK ? p.b[i] : p.a[i];
        if (row >= 0 && row < s.rows) atomicMin(&first[row], i);
    }
    __syncthreads();
    int asked = 0;
    for (int i0 = 0; i0 < p.n; i0 += kPlanThreads) {
        const int i = i0 + tid;
        Plan q = {-1, -1, -1, 0, 0, -1, -1, 0};
        if (i < p.n) {
            q.row = FORK ? p.b[i] : p.a[i];
            if (q.row >= 0 && q.row < s.rows && first[q.row] == i) {
                if (FORK) {
                    q.from = p.a[i];
                    if (q.from >= 0 && q.from < s.rows && q.from != q.row && s.lens[q.row] <= 0) {
                        q.len = row_len(s, q.from);
                        q.tail = q.len % s.page_size;
                        q.need = q.tail > 0;
                    }
                } else {
                    const int len = row_len(s, q.row), more = p.b[i];
                    if (more >= 0 && (long long)len + more <= (long long)s.cols * s.page_size) {
                        q.len = len;
                        q.need = pages_for(s, len + more) - pages_for(s, len);
                        q.tail = more;
                    }
                }
            }
        }
        int total;
        q.first = asked + scan(q.need, total) - q.need;
        asked += total;
        if (i < p.n) p.plan[i] = q;
    }
    const int got = free_pages(s, asked, is_free, p.list, scan);
    // all lengths and lists have been read: lengths may change now, and `done` may lie where a list does
    for (int i = tid; i < p.n; i += kPlanThreads) {
        Plan q = p.plan[i];
        const bool ok = q.len >= 0 && (q.need == 0 || q.first + q.need <= got);
        p.done[i] = ok;
        if (FORK) {
            if (ok) {
                s.lens[q.row] = q.len;
                if (q.need) {
                    const int at = q.len / s.page_size, src = s.table[(size_t)q.from * s.cols + at];
                    const int page = p.list[q.first];
                    s.table[(size_t)q.row * s.cols + at] = page;
                    s.refs[page] = 1;
                    q.src = src;
                    q.dst = in_pool(s, src) ? page : -1;
                }
            } else {
                q.len = -1;
                q.dst = -1;
            }
            p.plan[i] = q;
        } else if (ok) {
            s.lens[q.row] = q.len + q.tail;
        }
    }
    if (!FORK) {
        // a warp an item, a page a lane
        for (int i = tid >> 5; i < p.n; i += kPlanThreads / 32) {
            const Plan q = p.plan[i];
            if (q.len < 0 || q.first + q.need > got) continue;
            const int begin = pages_for(s, q.len);
            for (int k = tid & 31; k < q.need; k += 32) {
                const int page = p.list[q.first + k];
                s.table[(size_t)q.row * s.cols + begin + k] = page;
                s.refs[page] = 1;
            }
        }
    }
}

// ---------------------------------------------------------------- copies

constexpr int kCopyThreads = 256;

struct CopyCaches {
    const dl_kv_cache* at;   // on the device
    int n, heads, dim, block;
};

// One head's `tokens` first tokens of a page, keys or values, by a warp.
__device__ __forceinline__ void copy_head(const CopyCaches& c, int cache, int kv, int head, int src, int dst, int tokens) {
    const int lane = threadIdx.x & 31;
    const dl_kv_cache& k = c.at[cache];
    char* codes = static_cast<char*>(kv ? k.v : k.k) + head * k.head_stride;
    float* scales = (kv ? k.v_scale : k.k_scale) + head * k.scale_head_stride;
    const char* from = codes + src * k.page_stride;
    char* to = codes + dst * k.page_stride;
    const int bytes = tokens * c.dim;    // a multiple of 64
    const int blocks = (tokens + c.block - 1) / c.block;
    const float* sf = scales + src * k.scale_page_stride;
    float* st = scales + dst * k.scale_page_stride;
    for (int i = lane; i < blocks; i += 32) st[i] = sf[i];
    constexpr int kGroup = 8;            // 16-byte loads in flight
    for (int b0 = 16 * lane; b0 < bytes; b0 += 512 * kGroup) {
        uint4 v[kGroup];
#pragma unroll
        for (int k = 0; k < kGroup; ++k)
            if (b0 + 512 * k < bytes) v[k] = ldg128(from + b0 + 512 * k);
#pragma unroll
        for (int k = 0; k < kGroup; ++k)
            if (b0 + 512 * k < bytes) *reinterpret_cast<uint4*>(to + b0 + 512 * k) = v[k];
    }
}

struct ForkParams {
    PageState s;
    const Plan* plan;
    int n;
};

// The forked rows' tables, the counts of the pages that they share, and their begun pages' contents, in all caches
// at once: a warp copies a head's keys or values, eight loads in flight a lane.  Bound by these copies (101 MB both
// ways in 18 us, half of it DRAM's: what is written stays in L2).
__global__ void __launch_bounds__(kCopyThreads) fork_copy_kernel(const __grid_constant__ ForkParams p,
                                                                 const __grid_constant__ CopyCaches c) {
    griddep_wait();
    griddep_launch_dependents();
    const PageState& s = p.s;
    const int lane = threadIdx.x & 31;
    const long long warp = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5, warps = ((long long)gridDim.x * blockDim.x) >> 5;
    for (long long i = warp; i < p.n; i += warps) {
        const Plan q = p.plan[i];
        if (q.len < 0) continue;
        const int full = q.len / s.page_size;
        for (int k = lane; k < full; k += 32) {
            const int page = s.table[(size_t)q.from * s.cols + k];
            s.table[(size_t)q.row * s.cols + k] = page;
            if (in_pool(s, page)) atomicAdd(&s.refs[page], 1);
        }
    }
    const long long units = (long long)p.n * c.n * 2 * c.heads;
    for (long long u = warp; u < units; u += warps) {
        const int head = (int)(u % c.heads), kv = (int)(u / c.heads) & 1;
        const int cache = (int)(u / (2 * c.heads) % c.n);
        const Plan& q = p.plan[u / (2LL * c.heads * c.n)];
        if (q.dst >= 0) copy_head(c, cache, kv, head, q.src, q.dst, q.tail);
    }
}

struct CompactParams {
    PageState s;
    int *head;             // moves, pages in use
    int *src, *dst, *to;   // the moves; where a page at or past the used ones went
    int* live;
};

// Pages in use from the front on: those past the first `live` places move, in order, into the free
// places before it.  One CTA.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const __grid_constant__ CompactParams p) {
    __shared__ int warp_sum[2][32];
    Scan scan{warp_sum};
    const PageState& s = p.s;
    const int tid = threadIdx.x;
    griddep_wait();
    griddep_launch_dependents();
    int live = 0;
    for (int p0 = 0; p0 < s.num_pages; p0 += 16 * kPlanThreads) {
        int n = 0, total;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int page = p0 + k * kPlanThreads + tid;
            n += page < s.num_pages && s.refs[page] > 0;
        }
        scan(n, total);
        live += total;
    }
    int holes = 0, moves = 0;
    for (int p0 = 0; p0 < s.num_pages; p0 += 16 * kPlanThreads) {
        const int page0 = p0 + 16 * tid;
        unsigned hole = 0, move = 0;
        for (int k = 0; k < 16; ++k) {
            const int page = page0 + k;
            if (page >= s.num_pages) break;
            const bool used = s.refs[page] > 0;
            if (!used && page < live) hole |= 1u << k;
            if (used && page >= live) move |= 1u << k;
            if (!used && page >= live) p.to[page] = page;
        }
        int total;
        const int nh = __popc(hole), nm = __popc(move);
        int at = holes + scan(nh, total) - nh;
        holes += total;
        for (; hole; hole &= hole - 1) p.dst[at++] = page0 + __ffs(hole) - 1;
        at = moves + scan(nm, total) - nm;
        moves += total;
        for (; move; move &= move - 1) p.src[at++] = page0 + __ffs(move) - 1;
    }
    __syncthreads();
    for (int i = tid; i < moves; i += kPlanThreads) {
        const int src = p.src[i], dst = p.dst[i];
        p.to[src] = dst;
        s.refs[dst] = s.refs[src];
        s.refs[src] = 0;
    }
    if (tid == 0) {
        p.head[0] = moves;
        p.head[1] = live;
        p.live[0] = live;
    }
}

// The moves' contents in all caches, and the tables: memory bounds it (1.08 GB both ways in 158 us).
__global__ void __launch_bounds__(kCopyThreads) compact_copy_kernel(const __grid_constant__ CompactParams p,
                                                                    const __grid_constant__ CopyCaches c) {
    griddep_wait();
    griddep_launch_dependents();
    const PageState& s = p.s;
    const long long thread = (long long)blockIdx.x * blockDim.x + threadIdx.x, threads = (long long)gridDim.x * blockDim.x;
    const int moves = p.head[0], live = p.head[1];
    if (moves == 0) return;
    for (long long i = thread; i < (long long)s.rows * s.cols; i += threads) {
        if ((int)(i % s.cols) >= pages_for(s, row_len(s, (int)(i / s.cols)))) continue;
        const int page = s.table[i];
        if (page >= live && page < s.num_pages) s.table[i] = p.to[page];
    }
    const long long units = (long long)moves * c.n * 2 * c.heads;
    for (long long u = thread >> 5; u < units; u += threads >> 5) {
        const int head = (int)(u % c.heads), kv = (int)(u / c.heads) & 1;
        const int cache = (int)(u / (2 * c.heads) % c.n);
        const long long i = u / (2LL * c.heads * c.n);
        copy_head(c, cache, kv, head, p.src[i], p.dst[i], s.page_size);
    }
}

// ---------------------------------------------------------------- host

static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

static size_t pages_bytes(int num_pages, int rows) {
    return DL_WORKSPACE_ZERO_BYTES + 256 + up256((size_t)rows * sizeof(Plan)) + 3 * up256((size_t)num_pages * 4);
}

static dl_status check_pages(const dl_kv_pages* g, bool caches, PageState& s) {
    if (!g) return host_fail(DL_ERR_INVALID_ARG, "pages is NULL");
    if (g->num_pages < 1 || g->num_pages > (1 << 28))
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "num_pages=%d is outside [1, 2^28]", g->num_pages);
    if (g->page_size < 8 || g->page_size > 1024 || (g->page_size & (g->page_size - 1)))
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "page_size=%d is not a power of two in [8, 1024]", g->page_size);
    if (g->rows < 1 || g->rows > kMaxRows)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "rows=%d is outside [1, %d]", g->rows, kMaxRows);
    if (g->table_cols < 1) return host_fail(DL_ERR_INVALID_ARG, "table_cols=%d must be >= 1", g->table_cols);
    if ((long long)g->table_cols * g->page_size > 0x7fffffffLL)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "a row of %d pages of %d tokens exceeds 2^31 - 1", g->table_cols, g->page_size);
    // (what a list asks for is counted in 31 bits)
    if ((long long)g->rows * g->table_cols > 0x7fffffffLL)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "a table of %d x %d pages exceeds 2^31 - 1", g->rows, g->table_cols);
    if (!g->refs || !g->block_table || !g->seq_lens)
        return host_fail(DL_ERR_INVALID_ARG, "refs, block_table or seq_lens is NULL");
    if (((uintptr_t)g->refs | (uintptr_t)g->block_table | (uintptr_t)g->seq_lens) & 3)
        return host_fail(DL_ERR_MISALIGNED, "refs, block_table and seq_lens must be 4-byte aligned");
    if (g->num_caches < 0 || (g->num_caches && (!g->caches || (caches && !g->device_caches))))
        return host_fail(DL_ERR_INVALID_ARG, "caches or device_caches is NULL or num_caches=%d negative", g->num_caches);
    if (caches && ((uintptr_t)g->device_caches & 7)) return host_fail(DL_ERR_MISALIGNED, "device_caches must be 8-byte aligned");
    for (int i = 0; caches && i < g->num_caches; ++i) {
        const dl_kv_cache &c = g->caches[i], &c0 = g->caches[0];
        const dl_status st = check_cache(&c);
        if (st != DL_OK) return st;
        if (c.num_pages != g->num_pages || c.page_size != g->page_size || c.num_heads != c0.num_heads ||
            c.head_dim != c0.head_dim || c.block != c0.block)
            return host_fail(DL_ERR_INVALID_ARG, "cache %d has another shape than the pool or cache 0", i);
    }
    s = PageState{g->refs, g->block_table, g->seq_lens, g->num_pages, g->page_size, g->rows, g->table_cols};
    return DL_OK;
}

static dl_status check_list(const dl_kv_pages* g, const int* a, const int* b, bool two, const int* done, bool has_done, int n) {
    if (n < 0 || n > g->rows) return host_fail(DL_ERR_INVALID_ARG, "n=%d is outside [0, rows=%d]", n, g->rows);
    if (n == 0) return DL_OK;
    if (!a || (two && !b) || (has_done && !done)) return host_fail(DL_ERR_INVALID_ARG, "a list or done is NULL");
    if (((uintptr_t)a | (uintptr_t)b | (uintptr_t)done) & 3)
        return host_fail(DL_ERR_MISALIGNED, "lists and done must be 4-byte aligned");
    return DL_OK;
}

struct PagesScratch {
    int* head;
    Plan* plan;
    int* list[3];
};

static dl_status pages_scratch(const dl_kv_pages* g, void* ws, size_t ws_bytes, PagesScratch& out) {
    if (!ws) return host_fail(DL_ERR_WORKSPACE, "workspace is NULL");
    if ((uintptr_t)ws & 255) return host_fail(DL_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    const size_t need = pages_bytes(g->num_pages, g->rows);
    if (ws_bytes < need) return host_fail(DL_ERR_WORKSPACE, "workspace has %zu bytes, %zu are needed", ws_bytes, need);
    char* at = static_cast<char*>(ws) + DL_WORKSPACE_ZERO_BYTES;
    out.head = reinterpret_cast<int*>(at);
    at += 256;
    out.plan = reinterpret_cast<Plan*>(at);
    at += up256((size_t)g->rows * sizeof(Plan));
    for (int*& l : out.list) {
        l = reinterpret_cast<int*>(at);
        at += up256((size_t)g->num_pages * 4);
    }
    return DL_OK;
}

static CopyCaches copy_caches(const dl_kv_pages* g) {
    if (!g->num_caches) return CopyCaches{nullptr, 0, 1, 64, 1};
    const dl_kv_cache& k = g->caches[0];
    return CopyCaches{g->device_caches, g->num_caches, k.num_heads, k.head_dim, k.block};
}

template <bool FORK>
static cudaError_t launch_plan(const ListParams& p, cudaStream_t stream) {
    const size_t smem = (size_t)p.s.rows * 4;
    const cudaError_t e = raise_smem<plan_kernel<FORK>>((size_t)kMaxRows * 4);
    if (e != cudaSuccess) return e;
    return launch_dependent(plan_kernel<FORK>, dim3(1), dim3(kPlanThreads), smem, stream, p);
}

}  // namespace dl

extern "C" size_t dl_kv_pages_workspace_bytes(int num_pages, int rows) {
    if (num_pages < 1 || num_pages > (1 << 28) || rows < 1 || rows > dl::kMaxRows) return 0;
    return dl::pages_bytes(num_pages, rows);
}

extern "C" dl_status dl_kv_free(const dl_kv_pages* pages, const int* rows, int n, void* stream) {
    using namespace dl;
    PageState s;
    dl_status st = check_pages(pages, false, s);
    if (st != DL_OK || (st = check_list(pages, rows, nullptr, false, nullptr, false, n)) != DL_OK) return st;
    if (n == 0) return host_ok();
    const cudaError_t e = launch_dependent(free_rows_kernel, dim3(n), dim3(128), 0, static_cast<cudaStream_t>(stream), s, rows);
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "kv_free launch: %s", cudaGetErrorString(e));
    return host_ok();
}

extern "C" dl_status dl_kv_reserve(const dl_kv_pages* pages, const int* rows, const int* tokens, int* done, int n,
                                   void* workspace, size_t ws_bytes, void* stream) {
    using namespace dl;
    PageState s;
    PagesScratch w;
    dl_status st = check_pages(pages, false, s);
    if (st != DL_OK || (st = check_list(pages, rows, tokens, true, done, true, n)) != DL_OK) return st;
    if (n == 0) return host_ok();
    if ((st = pages_scratch(pages, workspace, ws_bytes, w)) != DL_OK) return st;
    const ListParams p = {s, rows, tokens, done, n, w.plan, w.list[0]};
    const cudaError_t e = launch_plan<false>(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "kv_reserve launch: %s", cudaGetErrorString(e));
    return host_ok();
}

extern "C" dl_status dl_kv_fork(const dl_kv_pages* pages, const int* parents, const int* children, int* done, int n,
                                void* workspace, size_t ws_bytes, void* stream) {
    using namespace dl;
    PageState s;
    PagesScratch w;
    dl_status st = check_pages(pages, true, s);
    if (st != DL_OK || (st = check_list(pages, parents, children, true, done, true, n)) != DL_OK) return st;
    if (n == 0) return host_ok();
    if ((st = pages_scratch(pages, workspace, ws_bytes, w)) != DL_OK) return st;
    HostDevice dev;
    if ((st = host_device(dev)) != DL_OK) return st;
    const cudaStream_t stm = static_cast<cudaStream_t>(stream);
    const ListParams p = {s, parents, children, done, n, w.plan, w.list[0]};
    cudaError_t e = launch_plan<true>(p, stm);
    const CopyCaches c = copy_caches(pages);
    const ForkParams f = {s, w.plan, n};
    const long long warps = (long long)n * (c.n ? c.n * 2LL * c.heads : 1);
    const long long ctas = (warps + kCopyThreads / 32 - 1) / (kCopyThreads / 32), most = 8LL * dev.sm_count;
    if (e == cudaSuccess)
        e = launch_dependent(fork_copy_kernel, dim3((unsigned)(ctas < most ? ctas : most)), dim3(kCopyThreads), 0, stm, f, c);
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "kv_fork launch: %s", cudaGetErrorString(e));
    return host_ok();
}

extern "C" dl_status dl_kv_compact(const dl_kv_pages* pages, int* live, void* workspace, size_t ws_bytes, void* stream) {
    using namespace dl;
    PageState s;
    PagesScratch w;
    dl_status st = check_pages(pages, true, s);
    if (st != DL_OK) return st;
    if (!live) return host_fail(DL_ERR_INVALID_ARG, "live is NULL");
    if ((uintptr_t)live & 3) return host_fail(DL_ERR_MISALIGNED, "live must be 4-byte aligned");
    if ((st = pages_scratch(pages, workspace, ws_bytes, w)) != DL_OK) return st;
    HostDevice dev;
    if ((st = host_device(dev)) != DL_OK) return st;
    const cudaStream_t stm = static_cast<cudaStream_t>(stream);
    const CompactParams p = {s, w.head, w.list[0], w.list[1], w.list[2], live};
    cudaError_t e = launch_dependent(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stm, p);
    if (e == cudaSuccess)
        e = launch_dependent(compact_copy_kernel, dim3((unsigned)(8 * dev.sm_count)), dim3(kCopyThreads), 0, stm, p, copy_caches(pages));
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "kv_compact launch: %s", cudaGetErrorString(e));
    return host_ok();
}
