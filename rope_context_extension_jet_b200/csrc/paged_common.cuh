// paged_common.cuh -- shared by the paged-cache operators: problem descriptions,
// the codes of the device input word, and the work plan of the paged decode.
//
// Cache layout: pages [num_pages][Hkv][page_size][d]; table[b][p] is the page
// that holds rows [p page_size, (p + 1) page_size) of request b.  Row lengths
// and page numbers live on the device (no host copy is needed to launch), so
// what the host cannot check is checked by the kernels: an out-of-range value
// is never followed, its request or row is left out, and a code is recorded in
// the device input word that jetlong_device_status reports.
#pragma once

#include <mutex>

#include "jl_common.cuh"

namespace jl {

constexpr int kNoPage = JETLONG_NO_PAGE;  // table entry of rows that block_tables refused

constexpr int kMaxNodes = 64;  // drafted tokens per request: ancestors fit one 64-bit mask

constexpr int kMaxTableRequests = 8192;  // block_tables: 5 words of shared memory per request

// Codes of the device input word.
enum {
    kBadPage = 0x201,     // a page number outside [0, num_pages)
    kBadSlot = 0x202,     // a slot outside [-1, num_pages * page_size)
    kBadLength = 0x203,   // a negative length, or rows beyond the block table
    kBadRows = 0x204,     // row_start decreasing, outside the token rows, or more than max_nodes apart
    kBadParent = 0x205,   // a parent that does not precede its node
    kBadFreeList = 0x206, // free_count outside the list, or more pages given back than it holds
};

struct PagedProblem {
    const void *q, *kc, *vc;
    void* out;
    const int *table, *lens, *row_start, *parents;  // row_start / parents may be null
    int B, N, Hq, Hkv, group;
    int num_pages, page_size, page_shift, max_pages, max_nodes;
    int w0, w_pre;
    float scale_log2;
    RopeTurns turns;
    unsigned char* workspace;
    int* input_error;
    int* dev_error;
    long long wait_cycles;  // 0: the normal limit
    int inject;
};

struct TablesProblem {
    const int *lens, *grow, *release, *held, *free_count;
    int *table, *free_list, *lens_out, *held_out, *free_count_out, *slot_map, *row_start, *status;
    int B, max_pages, page_size, page_shift, num_pages, free_cap, n_rows;
    int* input_error;
};

struct AppendProblem {
    const void *k, *v;
    const int* slots;
    void *kc, *vc;
    int N, Hkv, row_bytes;               // row_bytes = d * element size
    long long k_token, k_head, v_token, v_head;  // input strides in bytes
    int num_pages, page_size, page_shift;
    int* input_error;
};

struct CommitProblem {
    void *kc, *vc;
    const int *table, *lens, *row_start, *parents, *last;
    int *lens_out, *n_accepted;
    int B, N, Hkv, row_bytes, num_pages, page_size, page_shift, max_pages, max_nodes;
    int* input_error;
};

// Per device, done once: `set` (a kernel's attributes, its occupancy) and the number it
// returns through *value.  Such calls cost as much as a launch.
struct PerDevice {
    std::mutex mu;
    bool known[64] = {};
    int value[64] = {};
    template <class F>
    cudaError_t get(int* out, F set)
    {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        std::lock_guard<std::mutex> lk(mu);
        if (!known[dev]) {
            if ((e = set(&value[dev], dev)) != cudaSuccess) return e;
            known[dev] = true;
        }
        *out = value[dev];
        return cudaSuccess;
    }
};

cudaError_t launch_block_tables(const TablesProblem& p, cudaStream_t s, int* nlaunch);
cudaError_t launch_cache_append(const AppendProblem& p, cudaStream_t s, int* nlaunch);
cudaError_t launch_tree_commit(const CommitProblem& p, cudaStream_t s, int* nlaunch);
size_t paged_workspace_bytes(int B, int Hq, int Hkv, int d, int max_nodes);
int paged_tc_rows(int rows);
size_t paged_tc_workspace(int rows, int d);
int paged_fp32_rows(int rows);
size_t paged_fp32_workspace(int rows, int d);
cudaError_t launch_decode_paged_fp32(const PagedProblem& p, int d, cudaStream_t s, int* grid);
cudaError_t launch_decode_paged_tc(const PagedProblem& p, int d, cudaStream_t s, int* grid);
cudaError_t launch_decode_paged(const PagedProblem& p, int d, jetlong_dtype dt, cudaStream_t s, int* nlaunch);

__device__ __forceinline__ void record_input(int* word, int code)
{
    if (word) atomicCAS(word, 0, code);
}

#ifdef __CUDACC__

// ---------------------------------------------------------------------------
// Work plan of the paged decode.
//
// One unit = (request, kv head, tile of RT query rows); query row r of a
// request is node r / group, head r % group of the kv head.  A unit visits its
// keys in tiles of KT as a list of items: for every group size g its nodes can
// have, the tiles that can hold remote pairs (rotated to floor(x / g)), then
// the tiles that can hold local pairs (exact positions).  A tile on the border
// is visited in both with complementary masks, so one online softmax takes
// both branches.  With g = 1 throughout both rotations agree and every pair
// counts as local.
//
// All items of all units form one line, cut into equal pieces of `per` items,
// one per CTA: no CTA waits for the longest request.  A unit that lies in one
// piece is written out at once; the pieces of the others leave partial softmax
// states in the workspace (slot 2 c for the piece of CTA c that continues a
// unit, 2 c + 1 for one that begins it) for the merge kernel.
struct SeqPlan {
    int L, T;        // committed rows and nodes (T = 0: nothing to do)
    int n0;          // first token row
    int gmin, ng;    // group sizes gmin .. gmin + ng - 1 have remote phases (ng may be 0)
    int nR;          // tiles [0, nR) of each remote phase
    int kE0, n;      // tiles [kE0, n) of the exact phase
    int w0;          // window (INT_MAX when g = 1 throughout)
    int items;       // per unit
    int row_tiles;
};

// The request's rows up to `row` were refused their pages: its table holds no page for
// the last of them.  (What a refused request's table held there before, some other
// request's page perhaps, is not attended or written.)
__device__ __forceinline__ bool no_room(const int* table, int b, int max_pages, int page_shift, int row)
{
    return __ldg(table + (size_t)b * max_pages + (row >> page_shift)) == kNoPage;
}

// Largest depth of a tree (a parent that does not precede its node counts as -1).
__device__ inline int tree_depth(const int* parents, int T)
{
    unsigned char d[kMaxNodes];
    int most = 0;
    for (int t = 0; t < T; ++t) {
        const int x = parents[t];
        d[t] = (unsigned char)(x >= 0 && x < t ? d[x] + 1 : 0);
        most = max(most, (int)d[t]);
    }
    return most;
}

template <int KT, int RT>
__device__ inline SeqPlan seq_plan(const PagedProblem& p, int b, bool report)
{
    SeqPlan s;
    int L = p.lens[b], a = b, T = L >= 0 ? 1 : 0;
    int bad = 0;
    if (p.row_start) {
        a = p.row_start[b];
        T = p.row_start[b + 1] - a;
        if (a < 0 || T < 0 || T > p.max_nodes || a > p.N - T) {
            bad = kBadRows;
            T = 0;
        } else if (T > 0 && L < 0) {
            bad = kBadLength;
        }
    }
    if (T > 0 && (long long)L + T > (long long)p.max_pages * p.page_size) bad = kBadLength;
    if (bad) {
        if (report) record_input(p.input_error, bad);
        T = 0;
    } else if (T > 0 && no_room(p.table, b, p.max_pages, p.page_shift, L + T - 1)) {
        T = 0;
    }
    s.L = L;
    s.T = T;
    s.n0 = a;
    if (T == 0) {
        s.gmin = 1;
        s.ng = s.nR = s.kE0 = s.n = s.items = s.row_tiles = 0;
        s.w0 = 0;
        return s;
    }
    const int g0 = L / p.w_pre + 1;
    int imax = L + T - 1;  // no node is deeper than T - 1
    int g1 = imax / p.w_pre + 1;
    if (g1 > g0 && p.parents) {
        // a chain would cross into the next group size: the tree may not
        imax = L + tree_depth(p.parents + a, T);
        g1 = imax / p.w_pre + 1;
    }
    s.n = (L + T + KT - 1) / KT;
    s.gmin = g0;
    s.w0 = p.w0;
    if (g1 == 1) s.w0 = 0x7fffffff;
    // a tile can hold remote pairs if its smallest position is at most imax - w0
    // (drafted rows sit at positions >= L whatever their row)
    const int far = imax - s.w0;  // may be negative
    s.nR = far < 0 ? 0 : (far >= L ? s.n : min(s.n, far / KT + 1));
    s.ng = s.nR > 0 ? g1 - g0 + 1 : 0;
    // ... and local pairs if its largest position is at least L - w0 + 1
    if (s.w0 == 0) {
        s.kE0 = s.n;
    } else {
        const int lo = L - s.w0 + 1;
        s.kE0 = lo <= 0 ? 0 : min(lo / KT, s.n);
    }
    s.items = s.ng * s.nR + (s.n - s.kE0);
    s.row_tiles = (T * p.group + RT - 1) / RT;
    return s;
}

// Workspace: one CutUnit per CTA (the unit its piece begins and does not end, if
// any), then two partial states per CTA.
struct CutUnit {
    int rows;        // 0: none
    int pieces;      // CTAs c, c + 1, ... c + pieces - 1 hold it
    int node0, head0, r0;  // token row of the request's first node, first query head, first row of the unit
    int pad[3];
};
constexpr size_t kPagedHeader = 512 * sizeof(CutUnit);

// Whole-CTA: running sum of the requests' item counts; returns through shared
// memory the piece [start, end) of this CTA, the request it starts in and that
// request's first item.
struct PiecePlan {
    long long start, end, base, per;
    int b;
    SeqPlan first;  // plan of request b
};

// x / y; 64-bit division only where it is needed.
__device__ __forceinline__ long long quotient(long long x, long long y)
{
    if (x <= 0xffffffffll && y <= 0xffffffffll) return (long long)((unsigned)x / (unsigned)y);
    return x / y;
}

template <int KT, int RT, int NTHR>
__device__ void piece_plan(const PagedProblem& p, int min_items, PiecePlan* out, long long* scratch /* [NTHR/32] */)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int each = (p.B + NTHR - 1) / NTHR;
    const int b0 = min(p.B, tid * each), b1 = min(p.B, b0 + each);
    long long mine = 0;
    SeqPlan own;  // of request b0, for most threads their only one
    for (int b = b0; b < b1; ++b) {
        const SeqPlan s = seq_plan<KT, RT>(p, b, blockIdx.x == 0);
        mine += (long long)s.items * s.row_tiles * p.Hkv;
        if (b == b0) own = s;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < NTHR / 32; ++w) {
        const long long x = scratch[w];
        if (w < warp) before += x;
        total += x;
    }
    long long at = before + incl - mine;  // first item of this thread's requests
    long long per = quotient(total + gridDim.x - 1, gridDim.x);
    if (per < min_items) per = min_items;
    const long long start = min(total, per * blockIdx.x), end = min(total, start + per);
    if (tid == 0) {
        out->start = start;
        out->end = end;
        out->per = per;
    }
    if (start < end && at <= start && start < at + mine) {
        for (int b = b0; b < b1; ++b) {
            const SeqPlan s = b == b0 ? own : seq_plan<KT, RT>(p, b, false);
            const long long c = (long long)s.items * s.row_tiles * p.Hkv;
            if (at <= start && start < at + c) {
                out->b = b;
                out->base = at;
                out->first = s;
            }
            at += c;
        }
    }
    __syncthreads();
}

// Record of the unit this CTA's piece begins and does not end.  One thread per CTA
// writes it before the walk ends; a CTA that cuts no unit so leaves rows = 0.
__device__ __forceinline__ void clear_cut(const PagedProblem& p)
{
    reinterpret_cast<CutUnit*>(p.workspace)[blockIdx.x].rows = 0;
}
__device__ __forceinline__ void note_cut(const PagedProblem& p, const SeqPlan& s, long long per, long long first, int kvh,
                                         int r0, int rows)
{
    CutUnit* c = reinterpret_cast<CutUnit*>(p.workspace) + blockIdx.x;
    c->rows = rows;
    c->pieces = (int)(quotient(first + s.items - 1, per) - quotient(first, per) + 1);
    c->node0 = s.n0;
    c->head0 = kvh * p.group;
    c->r0 = r0;
}

// Quotient and remainder of a unit's place by its items; 64-bit division only
// where it is needed.
__device__ __forceinline__ void div_items(long long x, int items, int* q, int* r)
{
    if (x <= 0xffffffffll) {
        *q = (int)((unsigned)x / (unsigned)items);
        *r = (int)((unsigned)x % (unsigned)items);
    } else {
        *q = (int)(x / items);
        *r = (int)(x % items);
    }
}

#endif  // __CUDACC__

}  // namespace jl
