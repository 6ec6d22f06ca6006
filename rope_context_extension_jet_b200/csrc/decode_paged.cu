// decode_paged.cu -- bifocal decode over a paged raw-key cache, for one new token
// or a tree of drafted tokens per request: the fp32 kernel, the merge of split
// units, and the dispatch.
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

constexpr int PS_NT = 256, PS_KT = 64;
constexpr int kSimtCtas = 444;  // 3 per SM

namespace {

template <typename T> __device__ __forceinline__ float4 load4(const T* p);
template <> __device__ __forceinline__ float4 load4<float>(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <> __device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p)
{
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
}

template <int D, int RT>
struct SimtCfg {
    static constexpr int KR = 0;                           // [KT][D] rotated keys
    static constexpr int V = KR + PS_KT * D * 4;           // [KT][D] values
    static constexpr int Q = V + PS_KT * D * 4;            // [RT][D] rotated queries, base-2 logit units
    static constexpr int P = Q + RT * D * 4;               // [RT][KT] logits, then weights
    static constexpr int ML = P + RT * PS_KT * 4;          // [RT] max, sum, alpha
    static constexpr int ROW = ML + 3 * RT * 4;            // [RT] position, group size
    static constexpr int KPOS = ROW + 2 * RT * 4;          // [KT] key positions (-1: absent)
    static constexpr int ANC = KPOS + PS_KT * 4;           // [64] ancestors
    static constexpr int DEPTH = ANC + kMaxNodes * 8;
    static constexpr int PAR = DEPTH + kMaxNodes * 4;
    static constexpr int PLAN = PAR + kMaxNodes * 4;
    static constexpr int END = PLAN + (int)sizeof(PiecePlan) + 8 * (PS_NT / 32 + 1);
};

// Simple fp32 arithmetic on CUDA cores, so that fp32 inputs keep fp32 accuracy
// (TF32 would not).  A tile of KT keys is rotated once into shared memory and
// serves the RT query rows of the unit in groups of eight.
//   logits: 16 threads share a key quartet, each with 1/16 of the head
//     dimension (8 rows x 4 keys per thread in registers, then a halving
//     exchange over the 16 lanes);
//   P V: a thread holds 4 columns of all RT rows and takes every (NT / (D / 4))th key.
template <typename T, int D, int RT>
__global__ void __launch_bounds__(PS_NT, RT <= 8 ? 2 : 1) decode_paged_simt_kernel(PagedProblem p)
{
    using C = SimtCfg<D, RT>;
    constexpr int H = D / 2, NV = D / 64;
    constexpr int CG = D / 4, KS = PS_NT / CG;  // column groups, key slices of P V
    extern __shared__ __align__(16) unsigned char smem[];
    float* kr = reinterpret_cast<float*>(smem + C::KR);
    float* vs = reinterpret_cast<float*>(smem + C::V);
    float* qs = reinterpret_cast<float*>(smem + C::Q);
    float* ps = reinterpret_cast<float*>(smem + C::P);
    float* sm = reinterpret_cast<float*>(smem + C::ML);
    float *sl = sm + RT, *sa = sl + RT;
    int* qpos = reinterpret_cast<int*>(smem + C::ROW);
    int* qG = qpos + RT;
    int* kpos = reinterpret_cast<int*>(smem + C::KPOS);
    unsigned long long* anc = reinterpret_cast<unsigned long long*>(smem + C::ANC);
    int* depth = reinterpret_cast<int*>(smem + C::DEPTH);
    int* par = reinterpret_cast<int*>(smem + C::PAR);
    PiecePlan* plan = reinterpret_cast<PiecePlan*>(smem + C::PLAN);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    piece_plan<PS_KT, RT, PS_NT>(p, 2, plan, reinterpret_cast<long long*>(plan + 1));
    if (tid == 0) clear_cut(p);
    long long cur = plan->start, base = plan->base;
    const long long end = plan->end;
    int b = plan->b;
    const T* kc = static_cast<const T*>(p.kc);
    const T* vc = static_cast<const T*>(p.vc);
    const int slice = lane & 15, kg = tid >> 4;  // logits: 16 slices x 16 key groups
    const int col = (tid % CG) * 4, ks = tid / CG;

    while (cur < end) {
        SeqPlan s = seq_plan<PS_KT, RT>(p, b, false);
        long long cnt = (long long)s.items * s.row_tiles * p.Hkv;
        while (cur >= base + cnt) {
            base += cnt;
            ++b;
            s = seq_plan<PS_KT, RT>(p, b, false);
            cnt = (long long)s.items * s.row_tiles * p.Hkv;
        }
        int unit, i0;
        div_items(cur - base, s.items, &unit, &i0);
        const int i1 = (int)min((long long)s.items, i0 + (end - cur));
        const int kvh = unit / s.row_tiles, rt = unit % s.row_tiles;
        const int r0 = rt * RT, nrows = min(RT, s.T * p.group - r0);
        load_tree(p, s, par, depth, anc);
        for (int r = tid; r < RT; r += PS_NT) {
            int x = -1, G = 0;
            if (r < nrows) {
                x = s.L + depth[(r0 + r) / p.group];
                G = x / p.w_pre + 1;
            }
            qpos[r] = x;
            qG[r] = G;
            sm[r] = -INFINITY;
            sl[r] = 0.f;
        }
        float o[RT][4];
#pragma unroll
        for (int r = 0; r < RT; ++r) o[r][0] = o[r][1] = o[r][2] = o[r][3] = 0.f;
        int gcur = -1;
        Items item;
        item.start(s, i0);
        for (int it = i0; it < i1; ++it, item.next(s)) {
            const int g = item.g, tile = item.tile;
            __syncthreads();  // the previous tile is used up; qpos is ready
            if (g != gcur) {
                gcur = g;
                for (int e = tid; e < RT * H; e += PS_NT) {
                    const int r = e / H, m = e % H;
                    float x = 0.f, y = 0.f, c, sn;
                    if (r < nrows) {
                        const int node = (r0 + r) / p.group, hd = kvh * p.group + (r0 + r) % p.group;
                        const T* q = static_cast<const T*>(p.q) + ((size_t)(s.n0 + node) * p.Hq + hd) * D;
                        const float a = load_elem(q + m), bb = load_elem(q + m + H);
                        const uint32_t pos = g == 0 ? (uint32_t)qpos[r] : (uint32_t)qpos[r] / (uint32_t)g;
                        rope_cs_accurate(pos, p.turns.hi[m], p.turns.lo[m], c, sn);
                        x = (a * c - bb * sn) * p.scale_log2;
                        y = (a * sn + bb * c) * p.scale_log2;
                    }
                    qs[r * D + m] = x;
                    qs[r * D + m + H] = y;
                }
            }
            // keys rotated, values copied
#pragma unroll 2
            for (int e = tid; e < PS_KT * (H / 4); e += PS_NT) {
                const int kk = e / (H / 4), m = (e % (H / 4)) * 4;
                const int j = tile * PS_KT + kk;
                int pos = -1, page = -1;
                if (j < s.L + s.T) {
                    page = p.table[(size_t)b * p.max_pages + (j >> p.page_shift)];
                    pos = j < s.L ? j : s.L + depth[j - s.L];
                    if ((unsigned)page >= (unsigned)p.num_pages) {
                        record_input(p.input_error, kBadPage);
                        pos = -1;
                    }
                }
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f), c4 = a, va = a, vb = a;
                if (pos >= 0) {
                    const size_t at = (((size_t)page * p.Hkv + kvh) * p.page_size + (j & (p.page_size - 1))) * D;
                    a = load4(kc + at + m);
                    c4 = load4(kc + at + m + H);
                    va = load4(vc + at + m);
                    vb = load4(vc + at + m + H);
                    const uint32_t rp = g == 0 ? (uint32_t)pos : (uint32_t)pos / (uint32_t)g;
                    float* x = &a.x;
                    float* y = &c4.x;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        float c, sn;
                        rope_cs_accurate(rp, p.turns.hi[m + u], p.turns.lo[m + u], c, sn);
                        const float nx = x[u] * c - y[u] * sn;
                        y[u] = x[u] * sn + y[u] * c;
                        x[u] = nx;
                    }
                }
                *reinterpret_cast<float4*>(kr + kk * D + m) = a;
                *reinterpret_cast<float4*>(kr + kk * D + m + H) = c4;
                *reinterpret_cast<float4*>(vs + kk * D + m) = va;
                *reinterpret_cast<float4*>(vs + kk * D + m + H) = vb;
                if (m == 0) kpos[kk] = pos;
            }
            __syncthreads();
            for (int rg = 0; rg < RT; rg += 8) {
                if (rg >= nrows) break;
                float acc[32];  // [row of 8][key of 4]
#pragma unroll
                for (int x = 0; x < 32; ++x) acc[x] = 0.f;
#pragma unroll
                for (int v4 = 0; v4 < NV; ++v4) {
                    float4 kk[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        kk[i] = *reinterpret_cast<const float4*>(kr + (kg + 16 * i) * D + (slice + 16 * v4) * 4);
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float4 q4 = *reinterpret_cast<const float4*>(qs + (rg + r) * D + (slice + 16 * v4) * 4);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[r * 4 + i] = fmaf(q4.x, kk[i].x, fmaf(q4.y, kk[i].y, fmaf(q4.z, kk[i].z,
                                                  fmaf(q4.w, kk[i].w, acc[r * 4 + i]))));
                    }
                }
#pragma unroll
                for (int w = 16, bit = 8; w >= 2; w >>= 1, bit >>= 1) {
                    const bool hi = lane & bit;
#pragma unroll
                    for (int x = 0; x < w; ++x) {
                        const float give = hi ? acc[x] : acc[x + w], keep = hi ? acc[x + w] : acc[x];
                        acc[x] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
                    }
                }
                const int r = rg + (slice >> 1), x = qpos[r];
                const unsigned long long up = r < nrows ? anc[(r0 + r) / p.group] : 0ull;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int kk = kg + 16 * ((slice & 1) * 2 + i), pos = kpos[kk], u = tile * PS_KT + kk - s.L;
                    const bool local = x - pos < s.w0;
                    const bool keep = pos >= 0 && r < nrows && (u < 0 || ((up >> u) & 1)) &&
                                      (g == 0 ? local : (!local && qG[r] == g));
                    ps[r * PS_KT + kk] = keep ? acc[i] : -INFINITY;
                }
            }
            __syncthreads();
            for (int r = warp; r < nrows; r += PS_NT / 32) {
                const float a = ps[r * PS_KT + lane], c = ps[r * PS_KT + lane + 32];
                float mx = fmaxf(a, c);
                // a NaN logit is not a maximum, but its weight is NaN and stays in the sum
#pragma unroll
                for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
                const float m0 = sm[r], mn = fmaxf(m0, mx), ref = mn == -INFINITY ? 0.f : mn;
                const float wa = exp2f(a - ref), wc = exp2f(c - ref);
                float sum = wa + wc;
#pragma unroll
                for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
                ps[r * PS_KT + lane] = wa;
                ps[r * PS_KT + lane + 32] = wc;
                __syncwarp();
                if (lane == 0) {
                    const float alpha = exp2f(m0 - ref);
                    sa[r] = alpha;
                    sl[r] = sl[r] * alpha + sum;
                    sm[r] = mn;
                }
            }
            __syncthreads();
            // rows of drafted keys hide from nodes that do not descend from them:
            // a weight of 0 must not meet their infinities or NaN
            const bool drafted = (tile + 1) * PS_KT > s.L;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                if (r >= nrows) break;
                const float alpha = sa[r];
                o[r][0] *= alpha; o[r][1] *= alpha; o[r][2] *= alpha; o[r][3] *= alpha;
            }
            for (int kk = ks; kk < PS_KT; kk += KS) {
                const float4 v4 = *reinterpret_cast<const float4*>(vs + kk * D + col);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    if (r >= nrows) break;
                    const float w = ps[r * PS_KT + kk];
                    if (drafted && w == 0.f) continue;
                    o[r][0] = fmaf(w, v4.x, o[r][0]);
                    o[r][1] = fmaf(w, v4.y, o[r][1]);
                    o[r][2] = fmaf(w, v4.z, o[r][2]);
                    o[r][3] = fmaf(w, v4.w, o[r][3]);
                }
            }
        }
        // sum the key slices through shared memory, eight rows at a time, and write
        const bool whole = i0 == 0 && i1 == s.items;
        if (tid == 0 && i0 == 0 && !whole) note_cut(p, s, plan->per, cur, kvh, r0, nrows);
        float* part = reinterpret_cast<float*>(p.workspace + kPagedHeader) +
                      ((size_t)blockIdx.x * 2 + (i0 == 0 ? 1 : 0)) * RT * (D + 4);
        float* red = kr;  // [KS][8][D] = PS_NT * 32 floats: fits kr and vs together
#pragma unroll
        for (int rg = 0; rg < RT; rg += 8) {
            if (rg >= nrows) break;
            __syncthreads();
#pragma unroll
            for (int r = 0; r < 8; ++r)
                *reinterpret_cast<float4*>(red + (ks * 8 + r) * D + col) =
                    make_float4(o[rg + r][0], o[rg + r][1], o[rg + r][2], o[rg + r][3]);
            __syncthreads();
            for (int e = tid; e < 8 * D; e += PS_NT) {
                const int r = rg + e / D, c = e % D;
                if (r >= nrows) continue;
                float acc = 0.f;
                for (int w = 0; w < KS; ++w) acc += red[(w * 8 + e / D) * D + c];
                if (whole) {
                    const int node = (r0 + r) / p.group, hd = kvh * p.group + (r0 + r) % p.group;
                    store_elem(static_cast<T*>(p.out) + ((size_t)(s.n0 + node) * p.Hq + hd) * D + c, acc / sl[r]);
                } else {
                    part[(size_t)r * (D + 4) + c] = acc;
                    if (c < 2) part[(size_t)r * (D + 4) + D + c] = c == 0 ? sm[r] : sl[r];
                }
            }
        }
        __syncthreads();
        cur += i1 - i0;
    }
}

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

template <typename T, int D, int RT>
cudaError_t run_simt(const PagedProblem& p, cudaStream_t st, int* nlaunch)
{
    constexpr int smem = SimtCfg<D, RT>::END;
    static PerDevice once;
    int slots = 0;  // CTAs the device holds at a time
    cudaError_t e = once.get(&slots, [](int* n, int dev) {
        int nsm = 0, occ = 0;
        cudaError_t err = cudaFuncSetAttribute(decode_paged_simt_kernel<T, D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (err == cudaSuccess) err = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
        if (err == cudaSuccess)
            err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, decode_paged_simt_kernel<T, D, RT>, PS_NT, smem);
        *n = nsm * std::max(1, occ);
        return err;
    });
    if (e != cudaSuccess) return e;
    const int grid = std::min(kSimtCtas, slots);
    decode_paged_simt_kernel<T, D, RT><<<grid, PS_NT, smem, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    *nlaunch += 1;
    e = launch_after(decode_paged_merge_kernel<T, D, RT>, dim3(grid, merge_rows(p, RT)), MG_NT, st, p);
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
}

template <int D>
cudaError_t run_fp32(const PagedProblem& p, cudaStream_t st, int* nlaunch)
{
    if (p.max_nodes * p.group <= 8) return run_simt<float, D, 8>(p, st, nlaunch);
    return run_simt<float, D, 16>(p, st, nlaunch);
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
    const size_t simt = (size_t)kSimtCtas * 2 * (rows <= 8 ? 8 : 16) * (d + 4) * sizeof(float);
    return kPagedHeader + std::max(simt, paged_tc_workspace(rows, d));
}

cudaError_t launch_decode_paged(const PagedProblem& p, int d, jetlong_dtype dt, cudaStream_t s, int* nlaunch)
{
    if (dt == JETLONG_FP32) return d == 64 ? run_fp32<64>(p, s, nlaunch) : run_fp32<128>(p, s, nlaunch);
    return d == 64 ? run_bf16<64>(p, s, nlaunch) : run_bf16<128>(p, s, nlaunch);
}

}  // namespace jl
