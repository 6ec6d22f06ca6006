// paged_rows.cu -- rows moved into and within a paged cache: the append of new
// rows at their slots, and the commit of an accepted draft.  Both are plain
// copies (the cache holds unrotated rows, so a row keeps its value wherever it
// moves), bound by HBM bandwidth when large (append of 32,768 rows of 8 heads of 128 in
// bf16: 44 us, 6.1 TB/s read and written) and by one launch when small (16 rows: 3.3 us).
#include "paged_common.cuh"

namespace jl {
namespace {

constexpr int AP_NT = 256;
constexpr int AP_UNROLL = 4;  // 16-byte loads in flight per thread

// Row n, kv head h of k (v) goes to kcache (vcache) [slot / page_size][h][slot %
// page_size].  One thread moves 16 bytes of AP_UNROLL rows; a warp's chunks are
// consecutive, so reads and writes are whole rows.
__global__ void __launch_bounds__(AP_NT) cache_append_kernel(AppendProblem p)
{
    const int cpr = p.row_bytes >> 4;  // 16-byte chunks per row
    const long long total = (long long)p.N * p.Hkv * cpr;
    const bool is_v = blockIdx.y != 0;
    const char* src = static_cast<const char*>(is_v ? p.v : p.k);
    char* dst = static_cast<char*>(is_v ? p.vc : p.kc);
    const long long st = is_v ? p.v_token : p.k_token, sh = is_v ? p.v_head : p.k_head;
    const long long i0 = (long long)blockIdx.x * (AP_NT * AP_UNROLL) + threadIdx.x;
    uint4 x[AP_UNROLL];
    long long to[AP_UNROLL];
#pragma unroll
    for (int u = 0; u < AP_UNROLL; ++u) {
        const long long i = i0 + (long long)u * AP_NT;
        to[u] = -1;
        if (i >= total) continue;
        const int c = (int)(i % cpr);
        const long long rh = i / cpr;
        const int h = (int)(rh % p.Hkv), n = (int)(rh / p.Hkv);
        const int slot = __ldg(p.slots + n);
        if (slot < 0 || (slot >> p.page_shift) >= p.num_pages) {
            if (slot != -1) record_input(p.input_error, kBadSlot);
            continue;
        }
        const long long page = slot >> p.page_shift, off = slot & (p.page_size - 1);
        to[u] = ((page * p.Hkv + h) * p.page_size + off) * p.row_bytes + c * 16;
        x[u] = *reinterpret_cast<const uint4*>(src + n * st + h * sh + c * 16);
    }
#pragma unroll
    for (int u = 0; u < AP_UNROLL; ++u)
        if (to[u] >= 0) *reinterpret_cast<uint4*>(dst + to[u]) = x[u];
}

constexpr int CM_NT = 512;

// One CTA per request: the path is the ancestors-or-self of node `last`, in
// ascending order (a parent precedes its children), its row j moves from
// len + path[j] to len + j.  path[j] >= j, so with one thread moving a given
// 16-byte column of all path rows in order, no row is overwritten before it is read: a row
// below the current one is never read again, and loads of a group of rows come
// before its stores.  A request is committed whole or not at all: with a parent or a
// page out of range nothing of it moves and its length stays.
__global__ void __launch_bounds__(CM_NT) tree_commit_kernel(CommitProblem p)
{
    __shared__ int s_par[kMaxNodes], s_n;
    __shared__ long long s_src[kMaxNodes], s_dst[kMaxNodes];  // row offsets of kv head 0; source -1: stays where it is
    const int b = blockIdx.x, tid = threadIdx.x;
    const int L = p.lens[b];
    const int a = p.row_start[b];
    int T = p.row_start[b + 1] - a, last = p.last[b];
    int bad = 0;
    if (a < 0 || T < 0 || T > p.max_nodes || a > p.N - T) bad = kBadRows;
    else if (T > 0 && (L < 0 || (long long)L + T > (long long)p.max_pages * p.page_size)) bad = kBadLength;
    else if (last < -1 || last >= T) bad = kBadParent;
    if (bad && tid == 0) record_input(p.input_error, bad);
    if (bad || (T > 0 && no_room(p.table, b, p.max_pages, p.page_shift, L + T - 1))) {
        T = 0;
        last = -1;
    }
    bool wrong = false;
    if (tid < T) {
        int x = tid - 1;
        if (p.parents) {
            x = p.parents[a + tid];
            wrong = x < -1 || x >= tid;
            if (wrong) record_input(p.input_error, kBadParent);
        }
        s_par[tid] = x;
    }
    if (__syncthreads_or(wrong)) last = -1;
    if (tid == 0) {
        unsigned long long m = 0;
        for (int x = last; x >= 0; x = s_par[x]) m |= 1ull << x;
        int n = 0;
        for (; m; m &= m - 1) s_par[n++] = __ffsll((long long)m) - 1;  // n <= node: nothing still needed is overwritten
        s_n = n;
    }
    __syncthreads();
    int n = s_n;
    wrong = false;
    if (tid < n) {
        const int from = L + s_par[tid], to = L + tid;
        const int fp = p.table[(size_t)b * p.max_pages + (from >> p.page_shift)];
        const int tp = p.table[(size_t)b * p.max_pages + (to >> p.page_shift)];
        const bool ok = (unsigned)fp < (unsigned)p.num_pages && (unsigned)tp < (unsigned)p.num_pages;
        wrong = !ok;
        if (wrong) record_input(p.input_error, kBadPage);
        s_src[tid] = ok && from != to
                         ? ((long long)fp * p.Hkv * p.page_size + (from & (p.page_size - 1))) * p.row_bytes : -1;
        s_dst[tid] = ((long long)tp * p.Hkv * p.page_size + (to & (p.page_size - 1))) * p.row_bytes;
    }
    if (__syncthreads_or(wrong)) n = 0;
    const int cpr = p.row_bytes >> 4, cols = p.Hkv * cpr * 2;
    for (int c = tid; c < cols; c += CM_NT) {
        const int h = (c / cpr) % p.Hkv;
        char* base = static_cast<char*>(c >= p.Hkv * cpr ? p.vc : p.kc) +
                     (long long)h * p.page_size * p.row_bytes + (c % cpr) * 16;
        for (int j0 = 0; j0 < n; j0 += 8) {
            uint4 x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (j0 + u < n && s_src[j0 + u] >= 0) x[u] = *reinterpret_cast<const uint4*>(base + s_src[j0 + u]);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (j0 + u < n && s_src[j0 + u] >= 0) *reinterpret_cast<uint4*>(base + s_dst[j0 + u]) = x[u];
        }
    }
    if (tid == 0) {
        p.lens_out[b] = L + n;  // L of a request left out comes out as it went in
        if (p.n_accepted) p.n_accepted[b] = n;
    }
}

}  // namespace

cudaError_t launch_cache_append(const AppendProblem& p, cudaStream_t s, int* nlaunch)
{
    const long long chunks = (long long)p.N * p.Hkv * (p.row_bytes >> 4);
    const long long blocks = (chunks + AP_NT * AP_UNROLL - 1) / (AP_NT * AP_UNROLL);
    cache_append_kernel<<<dim3((unsigned)blocks, 2), AP_NT, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
}

cudaError_t launch_tree_commit(const CommitProblem& p, cudaStream_t s, int* nlaunch)
{
    tree_commit_kernel<<<p.B, CM_NT, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
}

}  // namespace jl
