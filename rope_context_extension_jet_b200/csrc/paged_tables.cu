// paged_tables.cu -- block tables and slot maps of a paged cache, from request
// lengths that live on the device.
//
// Request b holds held[b] pages for its lens[b] rows and takes grow[b] more rows:
//   need_b = max(0, ceil((lens_b + grow_b) / page_size) - held_b)  pages,
// granted in request order from the top of the free list while the running sum
// fits; the slot of new row o is table[b][(lens_b + o) / page_size] * page_size
// + (lens_b + o) % page_size.  Requests marked in `release` first give their
// pages back.
//
// A request that is refused (no pages left, or longer than its table row), idle or out of
// range takes no part; entries that its new rows would have needed become kNoPage, by
// which the other calls leave it out.
//
// All of it is prefix sums over requests and one store per row, so the call is
// bound by latency: one launch, no host copy.  Every CTA of one cluster scans
// all requests itself (three running sums in one pass) and then writes its share
// of the rows, each row finding its request by bisection of the row prefix in
// shared memory; one cluster barrier separates the pages given back, and every
// read of the old state, from the pages handed out and the new state, so inputs
// and outputs may be the same arrays.  (Pages of a table are read after the
// barrier only below held[b], where nothing is written.)
#include <limits.h>

#include "paged_common.cuh"
#include "jl_ptx.cuh"

namespace jl {
namespace {

constexpr int TB_NT = 512;
constexpr int kSmallRows = 4 * TB_NT;  // new rows that one CTA handles alone
// flags beside a page count (counts stay below 2^27): longer than its table row; numbers
// out of range, left as it is
constexpr int kLong = 1 << 30, kBad = 1 << 29;

struct Sum3 {
    long long rows;
    int need, back;
};

__device__ __forceinline__ Sum3 add3(const Sum3& a, const Sum3& b) { return {a.rows + b.rows, a.need + b.need, a.back + b.back}; }

struct Req {
    int len, grow, held, back, need;
    bool too_long, bad;
};

__device__ __forceinline__ Req load_req(const TablesProblem& p, int b, bool report)
{
    Req r;
    r.len = p.lens[b];
    r.grow = p.grow[b];
    r.held = p.held[b];
    r.back = 0;
    const bool released = p.release && p.release[b] != 0;
    r.need = 0;
    r.too_long = false;
    const bool idle = r.len < 0 && r.grow == 0;  // keeps its length, released or not
    r.bad = (r.len < 0 && !idle && !released) || r.grow < 0 || r.held < 0 || r.held > p.max_pages;
    if (r.bad) {
        if (report) record_input(p.input_error, kBadLength);
        r.grow = max(r.grow, 0);  // its token rows are counted
        r.held = 0;
        return r;
    }
    if (released) {
        r.back = r.held;
        r.held = 0;
        if (!idle) r.len = 0;
    }
    if (idle) return r;
    const long long pages = ((long long)r.len + r.grow + p.page_size - 1) >> p.page_shift;
    r.too_long = pages > p.max_pages;
    if (!r.too_long) r.need = max(0, (int)pages - r.held);
    return r;
}

// last index i in [0, n) with a[i] <= x (a[0] = 0 <= x)
__device__ __forceinline__ int bisect(const int* a, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// *to = the value made of *from and `off`
struct Move {
    const int* from;
    int* to;
    int off;
};

__global__ void __launch_bounds__(TB_NT) block_tables_kernel(TablesProblem p)
{
    // per request, read once before anything is written: running sums of rows,
    // pages needed and pages given back, rows held and pages held (both 0 once
    // released; kLong and kBad mark the requests that take no part)
    extern __shared__ int sm[];
    int* s_row = sm;
    int* s_need = s_row + p.B + 1;
    int* s_back = s_need + p.B + 1;
    int* s_len = s_back + p.B + 1;
    int* s_held = s_len + p.B + 1;
    __shared__ Sum3 s_warp[TB_NT / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x, gtid = cta * TB_NT + tid, gthr = gridDim.x * TB_NT;

    // For every x in [first, total), b the last index with sum[b] <= x: *to = value(*from,
    // off) of the Move f(x, b); to = null: nothing.  BATCH of them side by side: their
    // bisections and their loads overlap.
    auto each = [&](int first, int total, const int* sum, auto f, auto value) {
        constexpr int BATCH = 4;
        const int top = 1 << (31 - __clz(p.B));  // largest power of two <= B
#pragma unroll 1
        for (long long x0 = (long long)first + gtid; x0 < total; x0 += (long long)BATCH * gthr) {
            Move m[BATCH];
            int b[BATCH];
            bool in[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                b[u] = 0;
                in[u] = x0 + (long long)u * gthr < total;
            }
#pragma unroll 1
            for (int step = top; step > 0; step >>= 1) {
#pragma unroll
                for (int u = 0; u < BATCH; ++u) {
                    const int mid = min(b[u] + step, p.B - 1);
                    if (sum[mid] <= (in[u] ? (int)x0 + u * gthr : (int)x0)) b[u] = mid;
                }
            }
            int page[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                m[u] = f(in[u] ? (int)x0 + u * gthr : (int)x0, b[u]);
                if (!in[u]) m[u].to = nullptr;
            }
#pragma unroll
            for (int u = 0; u < BATCH; ++u) page[u] = m[u].to && m[u].from ? __ldcg(m[u].from) : -1;
#pragma unroll
            for (int u = 0; u < BATCH; ++u)
                if (m[u].to) *m[u].to = value(page[u], m[u].off);
        }
    };

    int count = *p.free_count;
    if (count < 0 || count > p.free_cap) {
        if (gtid == 0) record_input(p.input_error, kBadFreeList);
        count = min(max(count, 0), p.free_cap);
    }
    Sum3 carry = {0, 0, 0};
    for (int base = 0; base < p.B; base += TB_NT) {
        const int b = base + tid;
        Sum3 x = {0, 0, 0};
        if (b < p.B) {
            const Req r = load_req(p, b, cta == 0);
            x = {r.grow, r.need, r.back};
            s_len[b] = r.len;
            s_held[b] = r.held | (r.too_long ? kLong : 0) | (r.bad ? kBad : 0);
        }
        Sum3 incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            Sum3 up;
            up.rows = __shfl_up_sync(0xffffffffu, incl.rows, o);
            up.need = __shfl_up_sync(0xffffffffu, incl.need, o);
            up.back = __shfl_up_sync(0xffffffffu, incl.back, o);
            if (lane >= o) incl = add3(incl, up);
        }
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        Sum3 before = carry;
        for (int w = 0; w < TB_NT / 32; ++w) {
            const Sum3 y = s_warp[w];
            if (w < warp) before = add3(before, y);
            carry = add3(carry, y);
        }
        __syncthreads();
        if (b < p.B) {
            s_row[b] = (int)min((long long)INT_MAX, before.rows + incl.rows - x.rows);
            s_need[b] = before.need + incl.need - x.need;
            s_back[b] = before.back + incl.back - x.back;
        }
    }
    if (tid == 0) {
        s_row[p.B] = (int)min((long long)INT_MAX, carry.rows);
        s_need[p.B] = carry.need;
        s_back[p.B] = carry.back;
    }
    __syncthreads();
    if (gtid == 0 && carry.rows > p.n_rows) record_input(p.input_error, kBadRows);
    // pages given back: last request first, its last page first, so that pages
    // handed out together and given back together restore the list's order
    const auto checked = [&](int page, int) {  // what is no page is handed on as none
        if ((unsigned)page < (unsigned)p.num_pages) return page;
        record_input(p.input_error, kBadPage);
        return kNoPage;
    };
    if ((long long)count + carry.back > p.free_cap && gtid == 0) record_input(p.input_error, kBadFreeList);
    each(0, carry.back, s_back, [&](int x, int b) {
        const long long at = (long long)count + (carry.back - s_back[b + 1]) + (s_back[b + 1] - 1 - x);
        return Move{p.table + (size_t)b * p.max_pages + (x - s_back[b]), at < p.free_cap ? p.free_list + at : nullptr, 0};
    }, checked);
    // from here on the old state may be overwritten, and the list holds every free page
    cluster_sync();
    const int avail = (int)min((long long)p.free_cap, (long long)count + carry.back);
    // a request is granted if the running sum up to it fits; the sums ascend, so
    // the pages handed out are the largest sum that fits
    const int granted = s_need[bisect(s_need, p.B + 1, avail)];
    each(0, granted, s_need, [&](int x, int b) {
        return Move{p.free_list + (avail - 1 - x), p.table + (size_t)b * p.max_pages + s_held[b] + (x - s_need[b]), 0};
    }, checked);
    // the sums behind it are those of refused requests: their tables say so
    each(granted, s_need[p.B], s_need, [&](int x, int b) {
        return Move{nullptr, p.table + (size_t)b * p.max_pages + s_held[b] + (x - s_need[b]), 0};
    }, [](int, int) { return kNoPage; });
    for (int b = gtid; b < p.B; b += gthr) {
        const int need = s_need[b + 1] - s_need[b];
        const bool too_long = s_held[b] & kLong, refused = need > 0 && s_need[b + 1] > avail;
        const bool bad = s_held[b] & kBad;
        p.status[b] = bad ? 3 : too_long ? 2 : (refused ? 1 : 0);
        p.lens_out[b] = s_len[b];
        p.held_out[b] = bad ? p.held[b] : (s_held[b] & ~kLong) + (refused ? 0 : need);
        p.row_start[b] = s_row[b];
        if (bad && s_len[b] >= 0 && p.grow[b] > 0) {
            // what the table holds behind the committed rows is not to be followed either
            const int c = (int)(((long long)s_len[b] + p.grow[b] - 1) >> p.page_shift);
            if (c < p.max_pages && c > (s_len[b] - 1) >> p.page_shift) p.table[(size_t)b * p.max_pages + c] = kNoPage;
        }
    }
    if (gtid == 0) {
        p.row_start[p.B] = s_row[p.B];
        *p.free_count_out = avail - granted;
    }
    const int rows = min(p.n_rows, s_row[p.B]);
    each(0, rows, s_row, [&](int n, int b) {
        const int held = s_held[b], need = s_need[b], need1 = s_need[b + 1], pos = s_len[b] + (n - s_row[b]);
        const int c = pos >> p.page_shift;
        const int* from = c < held ? p.table + (size_t)b * p.max_pages + c : p.free_list + (avail - 1 - (need + c - held));
        if ((held & (kLong | kBad)) || (need1 > avail && need1 > need)) from = nullptr;  // takes no part, or refused
        return Move{from, p.slot_map + n, from ? pos & (p.page_size - 1) : -1};
    }, [&](int page, int off) {
        if (off < 0) return -1;
        if ((unsigned)page < (unsigned)p.num_pages) return (page << p.page_shift) + off;
        record_input(p.input_error, kBadPage);
        return -1;
    });
    for (long long n = (long long)rows + gtid; n < p.n_rows; n += gthr) p.slot_map[n] = -1;
}

}  // namespace

// One CTA where latency is all (B = 16, 16 rows: 5.1-5.5 us); else a cluster of eight
// (512 requests, 35,000 rows: 15.8 us; of 1024 threads each 19.4).
cudaError_t launch_block_tables(const TablesProblem& p, cudaStream_t s, int* nlaunch)
{
    static PerDevice once;
    int unused = 0;
    cudaError_t e = once.get(&unused, [](int*, int) {
        return cudaFuncSetAttribute(block_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    5 * (kMaxTableRequests + 1) * (int)sizeof(int));
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = p.n_rows <= kSmallRows ? 1 : 8;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.gridDim = dim3(at.val.clusterDim.x);
    cfg.blockDim = dim3(TB_NT);
    cfg.dynamicSmemBytes = 5 * (p.B + 1) * sizeof(int);
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, block_tables_kernel, p);
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
}

}  // namespace jl
