// decode_paged.cu -- bifocal decode over a paged raw-key cache, for one new token
// or a tree of drafted tokens per request: the mathematics, the merge of split units,
// and the dispatch (the kernels: decode_paged_fp32.cu, decode_paged_tc.cu,
// decode_paged_rows.cu).
//
// For node t of a request with len committed rows: position i = len + depth(t),
// G = max(1, ceil((i + 1) / w_pretrained)); it attends the committed rows j (at
// position j) and its ancestors-or-self u (row len + u, position len +
// depth(u)):
//   logit = <R(i) q, R(p) k>                     if i - p < w0,
//           <R(floor(i/G)) q, R(floor(p/G)) k>   otherwise,
//   out = sum_p softmax(scale logit)_p v_p.
// The work plan (paged_common.cuh) cuts all keys of all requests into equal
// pieces, one per CTA.
#include <algorithm>

#include "paged_common.cuh"

namespace jl {

namespace {

constexpr int MG_NT = 256, MG_SPLIT = 4, MG_ROWS = MG_NT / 32 / MG_SPLIT;

// Joins the pieces of every unit that was cut: out = sum_c 2^(m_c - M) o_c /
// sum_c 2^(m_c - M) l_c.  blockIdx.x is the CTA whose piece begins the unit (at
// most one such unit per CTA), blockIdx.y a pair of its rows; four warps share a
// row, each summing every fourth run of pieces in ascending order, so the result
// does not depend on which CTA finished first.
template <typename T, int D, int RT>
__global__ void __launch_bounds__(MG_NT) decode_paged_merge_kernel(PagedProblem p)
{
    constexpr int V = D / 32;  // columns per lane
    __shared__ float s_o[MG_NT / 32][D];
    __shared__ float s_m[MG_NT / 32], s_l[MG_NT / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const CutUnit* cut = reinterpret_cast<const CutUnit*>(p.workspace) + blockIdx.x;
    const int rows = __ldcg(&cut->rows), pieces = __ldcg(&cut->pieces);
    if ((int)blockIdx.y * MG_ROWS >= rows) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.y * MG_ROWS + warp / MG_SPLIT, sub = warp % MG_SPLIT;
    const float* parts = reinterpret_cast<const float*>(p.workspace + kPagedHeader);
    float M = -INFINITY, l = 0.f, o[V];
#pragma unroll
    for (int u = 0; u < V; ++u) o[u] = 0.f;
    // piece x: slot 2 c + 1 of the CTA that begins the unit, slot 2 (c + x) of the others
    auto piece = [&](int x) { return parts + ((size_t)(2 * (blockIdx.x + x) + (x == 0 ? 1 : 0)) * RT + r) * (D + 4); };
    if (r < rows) {
        const int each = (pieces + MG_SPLIT - 1) / MG_SPLIT, x1 = min(pieces, (sub + 1) * each);
        for (int x0 = sub * each; x0 < x1; x0 += 32) {
            // lane x holds the maximum and sum of piece x0 + x
            const int cnt = min(32, x1 - x0);
            float m = -INFINITY, ls = 0.f;
            if (lane < cnt) {
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(piece(x0 + lane) + D));
                m = ml.x;
                ls = ml.y;
            }
            float mx = m;
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float mn = fmaxf(M, mx), ref = mn == -INFINITY ? 0.f : mn;
            const float a = exp2f(M - ref), wgt = exp2f(m - ref);
            M = mn;
            float add = wgt * ls;
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) add += __shfl_xor_sync(0xffffffffu, add, w);
            l = l * a + add;
#pragma unroll
            for (int u = 0; u < V; ++u) o[u] *= a;
#pragma unroll 8
            for (int x = 0; x < cnt; ++x) {
                const float wx = __shfl_sync(0xffffffffu, wgt, x);
                const float* row = piece(x0 + x) + lane * V;
                if (wx != 0.f) {  // a piece without a key of this row holds no values
#pragma unroll
                    for (int u = 0; u < V; u += 2) {  // (lane * V: 8-byte aligned for d = 64)
                        const float2 v = __ldcg(reinterpret_cast<const float2*>(row + u));
                        o[u] = fmaf(wx, v.x, o[u]);
                        o[u + 1] = fmaf(wx, v.y, o[u + 1]);
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < V; ++u) s_o[warp][lane * V + u] = o[u];
        if (lane == 0) {
            s_m[warp] = M;
            s_l[warp] = l;
        }
    }
    __syncthreads();
    const int rr = threadIdx.x / (MG_NT / MG_ROWS), c = threadIdx.x % (MG_NT / MG_ROWS), row = blockIdx.y * MG_ROWS + rr;
    if (row >= rows || c >= D) return;
    float M4 = -INFINITY, num = 0.f, den = 0.f;
#pragma unroll
    for (int x = 0; x < MG_SPLIT; ++x) M4 = fmaxf(M4, s_m[rr * MG_SPLIT + x]);
    const float ref = M4 == -INFINITY ? 0.f : M4;
#pragma unroll
    for (int x = 0; x < MG_SPLIT; ++x) {
        const float w = exp2f(s_m[rr * MG_SPLIT + x] - ref);
        num = fmaf(w, s_o[rr * MG_SPLIT + x][c], num);
        den = fmaf(w, s_l[rr * MG_SPLIT + x], den);
    }
    const int r_unit = cut->r0 + row, node = cut->node0 + r_unit / p.group, hd = cut->head0 + r_unit % p.group;
    store_elem(static_cast<T*>(p.out) + ((size_t)node * p.Hq + hd) * D + c, num / den);
}

int merge_rows(const PagedProblem& p, int rt) { return (std::min(rt, p.max_nodes * p.group) + MG_ROWS - 1) / MG_ROWS; }

// Programmatic launch: the merge is set up while the attention kernel ends (an early
// trigger in that kernel gained 0.2 us of 18 on the smallest call and is left out).
template <class Kern>
cudaError_t launch_after(Kern kern, dim3 grid, int nthr, cudaStream_t st, const PagedProblem& p)
{
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(nthr);
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int D, int RT>
cudaError_t merge_fp32(const PagedProblem& p, int grid, cudaStream_t st)
{
    return launch_after(decode_paged_merge_kernel<float, D, RT>, dim3(grid, merge_rows(p, RT)), MG_NT, st, p);
}

template <int D>
cudaError_t run_fp32(const PagedProblem& p, cudaStream_t st, int* nlaunch)
{
    int grid = 0;
    cudaError_t e = launch_decode_paged_fp32(p, D, st, &grid);
    if (e != cudaSuccess) return e;
    *nlaunch += 1;
    switch (paged_fp32_rows(p.max_nodes * p.group)) {
        case 4: e = merge_fp32<D, 4>(p, grid, st); break;
        case 8: e = merge_fp32<D, 8>(p, grid, st); break;
        case 16: e = merge_fp32<D, 16>(p, grid, st); break;
        default: e = merge_fp32<D, 32>(p, grid, st); break;
    }
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
}

template <int D, int NCOL>
cudaError_t merge_tc(const PagedProblem& p, int grid, cudaStream_t st)
{
    return launch_after(decode_paged_merge_kernel<__nv_bfloat16, D, NCOL>, dim3(grid, merge_rows(p, NCOL)), MG_NT, st, p);
}

template <int D>
cudaError_t run_bf16(const PagedProblem& p, cudaStream_t st, int* nlaunch)
{
    int grid = 0;
    cudaError_t e = launch_decode_paged_tc(p, D, st, &grid);
    if (e != cudaSuccess) return e;
    *nlaunch += 1;
    switch (paged_tc_rows(p.max_nodes * p.group)) {
        case 16: e = merge_tc<D, 16>(p, grid, st); break;
        case 32: e = merge_tc<D, 32>(p, grid, st); break;
        case 128: e = merge_tc<D, 128>(p, grid, st); break;
        default: e = merge_tc<D, 256>(p, grid, st); break;
    }
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
}

}  // namespace

size_t paged_workspace_bytes(int B, int Hq, int Hkv, int d, int max_nodes)
{
    const int rows = max_nodes * (Hq / Hkv);
    return kPagedHeader + std::max(paged_fp32_workspace(rows, d), paged_tc_workspace(rows, d));
}

cudaError_t launch_decode_paged(const PagedProblem& p, int d, jetlong_dtype dt, cudaStream_t s, int* nlaunch)
{
    if (dt == JETLONG_FP32) return d == 64 ? run_fp32<64>(p, s, nlaunch) : run_fp32<128>(p, s, nlaunch);
    return d == 64 ? run_bf16<64>(p, s, nlaunch) : run_bf16<128>(p, s, nlaunch);
}

}  // namespace jl
