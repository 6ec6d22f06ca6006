// decode_paged_fp32.cu -- fp32 decode over a paged raw-key cache (mathematics and
// work plan: decode_paged.cu, paged_common.cuh), on the CUDA cores so that fp32
// inputs keep fp32 accuracy (TF32 products would not).
//
// A producer warp copies tiles of 32 keys and values (one bulk copy per page and
// operand; a page's rows of one head are contiguous) into a ring of NS stages; eight
// warps compute.  LPK lanes share a key, each with 4 + 4 of its dimensions (the two
// halves of 4 rotation pairs) of R query rows in registers, so a key is read from
// shared memory once per R rows:
//   rotation   4 pairs in registers; angles fresh for each run of 8 or 16 keys, inside it
//              by angle addition (at most 15 steps of 3 * 2^-24 each: below half of
//              what the products' 128 terms may round by)
//   logits     partial dots of KB = LPK / R keys, then a halving exchange that leaves
//              one (key, row) logit on each lane
//   softmax    the lane's running reference, moved only when a logit passes it by
//              2^16 (weights stay far inside fp32)
//   P V        weights by shuffle; 4 + 4 output columns per lane and row
// A unit of RT = R WR rows puts WR warps on every tile (a row group each) and spreads
// tiles over 8 / WR key groups; their states are joined where the unit ends.
//
// Bound: HBM up to 8 rows.  Measured, 32 query heads on 8, d = 128: 8 requests of 16,000
// rows 178 us (5.9 TB/s of K and V).  With more rows it is far from either bound: trees
// of 8 nodes on them 660-720 us, where the 256 FMA per key and row take 235.  Each row
// group of a unit turns every key again, and each (key, row) costs a shuffle for its
// weight and its part of the exchange of the dots.  (Without the next batch's logits
// beside this one's values 213 and 865 us; keys and values staged by plain loads 567
// and 2310.)
#include <algorithm>

#include "paged_common.cuh"
#include "prefill_tc_common.cuh"

namespace jl {

namespace {

constexpr int KT = 32;                  // keys of a tile
constexpr int CW = 8, CT = CW * 32;     // computing warps, threads
constexpr int NTHR = CT + 128;          // and the producer's warpgroup
// Registers per thread after setmaxnreg: the two computing warpgroups, the producer's
// (384 threads launch with 168 each, and an increase draws on that).
constexpr int R_CALC = 232, R_PROD = 40;
static_assert((2 * R_CALC + R_PROD) * 128 <= NTHR * 168, "register split");
constexpr int kCtas = 148;              // one per SM
constexpr int kMinItems = 4;            // tiles of a piece at least
constexpr float kExceed = 16.f;

template <int D, int RT>
struct Cfg {
    static constexpr int R = RT < 8 ? RT : 8, WR = RT / R, WK = CW / WR;
    static constexpr int LPK = D / 8, KB = LPK / R, NG = 32 / LPK, RUN = KT / NG;
    static constexpr int NS = (RT <= 4 ? 6 : 5) * (128 / D);
    // Landed tiles are announced on a ring of NB barriers, a multiple of the key groups:
    // each barrier belongs to one of them, which so sees all of its phases.
    static constexpr int NB = (NS + CW - 1) / CW * CW;
    static constexpr int TILE = KT * D * 4;
    static constexpr int V0 = NS * TILE;
    static constexpr int Q = 2 * V0;                       // [RT][D] rotated queries, base-2 logit units
    static constexpr int RED = Q + RT * D * 4;             // [CW][R][D] outputs of the warps
    static constexpr int ML = RED + CW * R * D * 4;        // [CW][R] (reference, sum)
    static constexpr int FULL = ML + CW * R * 8;
    static constexpr int EMPTY = FULL + NB * 8;
    static constexpr int ANC = EMPTY + NS * 8;
    static constexpr int DEPTH = ANC + kMaxNodes * 8;
    static constexpr int PAR = DEPTH + kMaxNodes * 4;
    static constexpr int NOTE = PAR + kMaxNodes * 4;       // [NS] mask of the pages present
    static constexpr int FLAG = NOTE + NS * 4;             // abort flag, no work
    static constexpr int PLAN = (FLAG + 8 + 15) / 16 * 16;
    static constexpr int SCAN = PLAN + (int)sizeof(PiecePlan);
    static constexpr int END = SCAN + (NTHR / 32) * 8;
    static_assert(LPK % R == 0 && CW % WR == 0 && NB >= NS && NB % WK == 0, "layout");
    static_assert(PLAN % 8 == 0 && SCAN % 8 == 0 && END <= 232448, "shared memory");
};

__device__ __forceinline__ void named_sync() { asm volatile("bar.sync 1, %0;" ::"n"(CT) : "memory"); }
__device__ __forceinline__ bool named_or(bool x)
{
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"((int)x), "n"(CT) : "memory");
    return r != 0;
}

// A CTA's piece, unit by unit.
template <int RT>
struct Walk {
    const PagedProblem& p;
    long long cur, base, end;
    int b, i0, i1, kvh, r0;
    SeqPlan s;
    __device__ __forceinline__ Walk(const PagedProblem& p_, const PiecePlan* plan, bool work)
        : p(p_), cur(plan->start), base(plan->base), end(work ? plan->end : plan->start), b(plan->b), s(plan->first) {}
    __device__ __forceinline__ bool unit()
    {
        if (cur >= end) return false;
        long long cnt = (long long)s.items * s.row_tiles * p.Hkv;
        while (cur >= base + cnt) {
            base += cnt;
            ++b;
            s = seq_plan<KT, RT>(p, b, false);
            cnt = (long long)s.items * s.row_tiles * p.Hkv;
        }
        int u;
        div_items(cur - base, s.items, &u, &i0);
        i1 = (int)min((long long)s.items, i0 + (end - cur));
        kvh = u / s.row_tiles;
        r0 = (u % s.row_tiles) * RT;
        return true;
    }
    __device__ __forceinline__ void done() { cur += i1 - i0; }
};
// A phase of a unit from item i on: the group size (0: exact positions), the first
// tile, and how many of the items before i1 belong to it.
__device__ __forceinline__ void phase_at(const SeqPlan& s, int i, int i1, int* g, int* tile, int* cnt)
{
    const int rem = s.ng * s.nR;
    *g = 0;
    *tile = s.kE0 + (i - rem);
    *cnt = i1 - i;
    if (i < rem) {
        *g = s.gmin + i / s.nR;
        *tile = i % s.nR;
        *cnt = min(*cnt, s.nR - *tile);
    }
}

template <int D, int RT>
__global__ void __launch_bounds__(NTHR, 1) decode_paged_fp32_kernel(const __grid_constant__ PagedProblem p, const long long wait_cycles)
{
    using C = Cfg<D, RT>;
    constexpr int R = C::R, H = D / 2, LPK = C::LPK, KB = C::KB;
    extern __shared__ __align__(128) unsigned char smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::FULL);
    uint64_t* empty = reinterpret_cast<uint64_t*>(smem + C::EMPTY);
    volatile unsigned* note = reinterpret_cast<volatile unsigned*>(smem + C::NOTE);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::FLAG);
    PiecePlan* plan = reinterpret_cast<PiecePlan*>(smem + C::PLAN);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == NTHR - 1) {  // (the first threads go on to the requests' lengths)
        for (int s = 0; s < C::NB; ++s) mbar_init(&full[s], 1);
        for (int s = 0; s < C::NS; ++s) mbar_init(&empty[s], C::WR);
        // an earlier wait ran out: no work
        abort_flag[0] = abort_flag[1] = *reinterpret_cast<volatile int*>(p.dev_error) != 0;
        fence_mbar_init();
        clear_cut(p);
    }
    // ends with a barrier of the CTA
    piece_plan<KT, RT, NTHR>(p, kMinItems, plan, reinterpret_cast<long long*>(smem + C::SCAN));
    Walk<RT> walk(p, plan, abort_flag[1] == 0);
    const SeqPlan& s = walk.s;
    int e = 0;  // items of the piece so far

    if (warp >= CW) {
        // ------------------------------------------------------ producer
        regs_dec<R_PROD>();
        if (warp != CW) return;
        const int box = min(p.page_size, KT), nbox = KT / box, ahead = 32 / nbox;
        bool ok = true;
        while (ok && walk.unit()) {
            const int* table = p.table + (size_t)walk.b * p.max_pages;
            const int n = s.L + s.T;
            for (int i = walk.i0; ok && i < walk.i1;) {
                int g, tile, cnt;
                phase_at(s, i, walk.i1, &g, &tile, &cnt);
                int pages = -1;  // lane x: page of box x of the tiles at hand
                for (int x = 0; x < cnt; ++x, ++e) {
                    if (x % ahead == 0) {
                        const int row = (tile + x) * KT + lane * box;
                        pages = -1;
                        if (x + lane / nbox < cnt && row < n) {
                            pages = __ldg(table + (row >> p.page_shift));
                            if ((unsigned)pages >= (unsigned)p.num_pages) {
                                record_input(p.input_error, kBadPage);
                                pages = -1;
                            }
                        }
                    }
                    const int page = __shfl_sync(0xffffffffu, pages, (x % ahead) * nbox + (lane < nbox ? lane : 0));
                    const unsigned have = __ballot_sync(0xffffffffu, lane < nbox && page >= 0);
                    const int st = e % C::NS;
                    if (e >= C::NS &&
                        !tc::warp_wait(&empty[st], ((e / C::NS) - 1) & 1, abort_flag, p.dev_error, wait_cycles, 0x701)) {
                        ok = false;
                        break;
                    }
                    if (e == 0 && p.inject == kInjectDecodeCopy) continue;  // test hook: the first tile is never loaded
                    uint64_t* bar = &full[e % C::NB];
                    if (lane == 0) {
                        note[st] = have;
                        if (have)
                            mbar_arrive_expect_tx(bar, (uint32_t)(__popc(have) * box * D * 8));
                        else
                            mbar_arrive(bar);
                    }
                    __syncwarp();
                    if (lane < nbox && page >= 0) {
                        const int row = (tile + x) * KT + lane * box;
                        const size_t at = (((size_t)page * p.Hkv + walk.kvh) * p.page_size + (row & (p.page_size - 1))) * D;
                        const int to = st * C::TILE + lane * box * D * 4;
                        bulk_g2s(smem + to, static_cast<const float*>(p.kc) + at, box * D * 4, bar);
                        bulk_g2s(smem + C::V0 + to, static_cast<const float*>(p.vc) + at, box * D * 4, bar);
                    }
                }
                i += cnt;
            }
            walk.done();
        }
        // the copies in flight land before the CTA ends
        for (int x = max(0, e - C::NS); x < e; ++x)
            if (!(x == 0 && p.inject == kInjectDecodeCopy)) mbar_wait(&full[x % C::NB], (x / C::NB) & 1);
        return;
    }

    // ---------------------------------------------------------- computing warps
    regs_inc<R_CALC>();
    float* qs = reinterpret_cast<float*>(smem + C::Q);
    float* red = reinterpret_cast<float*>(smem + C::RED);
    float2* ml = reinterpret_cast<float2*>(smem + C::ML);
    unsigned long long* anc = reinterpret_cast<unsigned long long*>(smem + C::ANC);
    int* depth = reinterpret_cast<int*>(smem + C::DEPTH);
    int* par = reinterpret_cast<int*>(smem + C::PAR);
    const int rg = warp % C::WR, kg = warp / C::WR;       // row group, key group
    const int sub = lane % LPK, grp = lane / LPK, m0 = sub * 4;  // dimensions m0 .. m0 + 3 and H + m0 ..
    const int shift = min(p.page_shift, 5);
    const unsigned all = KT >> shift >= 32 ? 0xffffffffu : (1u << (KT >> shift)) - 1;
    auto angles = [&](uint32_t f, float2 (&cs)[2], float2 (&sn)[2]) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            rope_cs_accurate(f, p.turns.hi[m0 + 2 * u], p.turns.lo[m0 + 2 * u], cs[u].x, sn[u].x);
            rope_cs_accurate(f, p.turns.hi[m0 + 2 * u + 1], p.turns.lo[m0 + 2 * u + 1], cs[u].y, sn[u].y);
        }
    };
    float2 stc[2], sts[2];  // one position further
    angles(1u, stc, sts);

    while (walk.unit()) {
        const int L = s.L, T = s.T, n = L + T, nrows = min(RT, T * p.group - walk.r0);
        if (named_or(false)) return;  // the last unit's notes are read
        if (tid < T) {
            int x = tid - 1;
            if (p.parents) {
                x = p.parents[s.n0 + tid];
                if (x < -1 || x >= tid) {
                    record_input(p.input_error, kBadParent);
                    x = -1;
                }
            }
            par[tid] = x;
        }
        named_sync();
        if (tid < T) {
            unsigned long long m = (2ull << tid) - 1;  // tid = 63: 2 << 63 is 0, so all ones
            if (p.parents) {
                m = 0;
                for (int x = tid; x >= 0; x = par[x]) m |= 1ull << x;
            }
            anc[tid] = m;
            depth[tid] = __popcll(m) - 1;
        }
        named_sync();
        // the row whose logits this lane holds
        const int row = rg * R + sub % R, rnode = (walk.r0 + row) / p.group;
        int lim = 0, G = 0;
        unsigned long long up = 0;
        if (row < nrows) {
            const int x = L + depth[rnode];
            lim = x - s.w0;
            G = x / p.w_pre + 1;
            up = anc[rnode];
        }
        const int near = n - 1 - s.w0;
        const int far = s.ng > 1 ? -1 : (int)max(-1ll, (long long)L - s.w0 - (KT - 1));
        float ref = -INFINITY, l = 0.f;
        float2 q[R][4], o[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int u = 0; u < 4; ++u) o[r][u] = make_float2(0.f, 0.f);
        bool ok = true;
        for (int i = walk.i0; i < walk.i1;) {
            int g, tile0, cnt;
            phase_at(s, i, walk.i1, &g, &tile0, &cnt);
            if (named_or(!ok)) return;  // and the last phase's queries are read
            for (int x = tid; x < RT * H; x += CT) {
                const int r = x / H, m = x % H;
                float a = 0.f, b = 0.f;
                if (r < nrows) {
                    const int node = (walk.r0 + r) / p.group, hd = walk.kvh * p.group + (walk.r0 + r) % p.group;
                    const float* src = static_cast<const float*>(p.q) + ((size_t)(s.n0 + node) * p.Hq + hd) * D;
                    const float qa = src[m], qb = src[m + H];
                    float c, sn;
                    rope_cs_accurate((uint32_t)(L + depth[node]) / (uint32_t)max(g, 1), p.turns.hi[m], p.turns.lo[m], c, sn);
                    a = (qa * c - qb * sn) * p.scale_log2;
                    b = (qa * sn + qb * c) * p.scale_log2;
                }
                qs[r * D + m] = a;
                qs[r * D + m + H] = b;
            }
            named_sync();
            // division by the group size by multiply-shift
            const uint32_t dv = max(g, 1), lg = 32 - __clz(dv - 1);  // ceil(log2 dv); 0 for 1
            const uint32_t dm = (uint32_t)(((((uint64_t)1 << 32) * (((uint64_t)1 << lg) - dv)) / dv) + 1);
            const uint32_t ds1 = min(lg, 1u), ds2 = lg > 1 ? lg - 1 : 0;
            auto over_g = [&](uint32_t pos) {
                const uint32_t t1 = __umulhi(dm, pos);
                return (t1 + ((pos - t1) >> ds1)) >> ds2;
            };
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float4 a = *reinterpret_cast<const float4*>(qs + (rg * R + r) * D + m0);
                const float4 b = *reinterpret_cast<const float4*>(qs + (rg * R + r) * D + m0 + H);
                q[r][0] = make_float2(a.x, a.y);
                q[r][1] = make_float2(a.z, a.w);
                q[r][2] = make_float2(b.x, b.y);
                q[r][3] = make_float2(b.z, b.w);
            }
            // this key group's tiles of the phase
            for (int x = (kg - e % C::WK + C::WK) % C::WK; x < cnt; x += C::WK) {
                const int ee = e + x, st = ee % C::NS, j0 = (tile0 + x) * KT;
                if (!tc::warp_wait(&full[ee % C::NB], (ee / C::NB) & 1, abort_flag, p.dev_error, wait_cycles, 0x711)) {
                    ok = false;
                    break;
                }
                const unsigned have = note[st];
                // rows that do not exist hold anything, drafted ones hide from nodes that do
                // not descend from them: a weight of 0 must not meet their infinities or NaN
                const bool risky = j0 + KT > L || have != all;
                const bool masked = risky || (g == 0 ? j0 <= near : j0 > far);
                const float* kt = reinterpret_cast<const float*>(smem + st * C::TILE) + grp * C::RUN * D + m0;
                const float* vt = reinterpret_cast<const float*>(smem + C::V0 + st * C::TILE) + grp * C::RUN * D + m0;
                const int jr = j0 + grp * C::RUN;
                uint32_t f = 0;
                float2 cs[2], sn[2];
                // Logit `sub` of the batch of keys from kk on: key kk + sub / R, row sub % R.
                // Within a run the turned position of row j, floor(j / g), stays or steps by one.
                auto logit = [&](int kk, bool fresh) {
                    float acc[LPK];
#pragma unroll
                    for (int b = 0; b < KB; ++b) {
                        const int j = jr + kk + b;
                        if (fresh) {
                            angles(over_g(j < L ? (uint32_t)j : j < n ? (uint32_t)(L + depth[j - L]) : 0u), cs, sn);
                        } else {
                            const uint32_t fn = over_g((uint32_t)j);
                            if (fn != f) {
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    const float2 nc = fma2(make_float2(-sn[u].x, -sn[u].y), sts[u], mul2(cs[u], stc[u]));
                                    sn[u] = fma2(cs[u], sts[u], mul2(sn[u], stc[u]));
                                    cs[u] = nc;
                                }
                            }
                            f = fn;
                        }
                        const float4 a = *reinterpret_cast<const float4*>(kt + (kk + b) * D);
                        const float4 c = *reinterpret_cast<const float4*>(kt + (kk + b) * D + H);
                        const float2 x0 = make_float2(a.x, a.y), x1 = make_float2(a.z, a.w);
                        const float2 y0 = make_float2(c.x, c.y), y1 = make_float2(c.z, c.w);
                        const float2 k0 = fma2(make_float2(-y0.x, -y0.y), sn[0], mul2(x0, cs[0]));
                        const float2 k1 = fma2(make_float2(-y1.x, -y1.y), sn[1], mul2(x1, cs[1]));
                        const float2 k2 = fma2(y0, cs[0], mul2(x0, sn[0]));
                        const float2 k3 = fma2(y1, cs[1], mul2(x1, sn[1]));
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const float2 d = fma2(q[r][3], k3, fma2(q[r][2], k2, fma2(q[r][1], k1, mul2(q[r][0], k0))));
                            acc[b * R + r] = d.x + d.y;
                        }
                    }
#pragma unroll
                    for (int w = LPK / 2; w >= 1; w >>= 1) {
                        const bool hi = lane & w;
#pragma unroll
                        for (int u = 0; u < w; ++u) {
                            const float give = hi ? acc[u] : acc[u + w], mine = hi ? acc[u + w] : acc[u];
                            acc[u] = mine + __shfl_xor_sync(0xffffffffu, give, w);
                        }
                    }
                    return acc[0];
                };
                // its weight; the reference moves where it has to
                auto weight = [&](float y, int kk) {
                    if (masked) {
                        const int kx = grp * C::RUN + kk + sub / R, j = j0 + kx, u = j - L;
                        const bool there = j < n && ((have >> (kx >> shift)) & 1) && row < nrows;
                        bool keep = false;
                        if (there) {
                            const bool local = (u < 0 ? j : L + depth[u]) > lim;
                            keep = (u < 0 || ((up >> u) & 1)) && (g == 0 ? local : (!local && G == g));
                        }
                        y = keep ? y : -INFINITY;
                    }
                    // a NaN logit is not a maximum, but its weight is NaN and stays in the sum
                    float mx = y;
#pragma unroll
                    for (int w = R; w < LPK; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
                    const bool move = mx > ref + kExceed;
                    if (__any_sync(0xffffffffu, move)) {
                        const float alpha = move ? exp2f(ref - mx) : 1.f;
                        ref = move ? mx : ref;
                        l *= alpha;
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const float a = __shfl_sync(0xffffffffu, alpha, r, LPK);
#pragma unroll
                            for (int u = 0; u < 4; ++u) o[r][u] = mul2(o[r][u], make_float2(a, a));
                        }
                    }
                    const float w = exp2f(y - (ref == -INFINITY ? 0.f : ref));
                    l += w;
                    return w;
                };
                auto values = [&](float w, int kk, bool guard) {
#pragma unroll
                    for (int b = 0; b < KB; ++b) {
                        const float4 a = *reinterpret_cast<const float4*>(vt + (kk + b) * D);
                        const float4 c = *reinterpret_cast<const float4*>(vt + (kk + b) * D + H);
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const float wr = __shfl_sync(0xffffffffu, w, b * R + r, LPK);
                            if (!guard || wr != 0.f) {
                                const float2 w2 = make_float2(wr, wr);
                                o[r][0] = fma2(w2, make_float2(a.x, a.y), o[r][0]);
                                o[r][1] = fma2(w2, make_float2(a.z, a.w), o[r][1]);
                                o[r][2] = fma2(w2, make_float2(c.x, c.y), o[r][2]);
                                o[r][3] = fma2(w2, make_float2(c.z, c.w), o[r][3]);
                            }
                        }
                    }
                };
                if (!risky) {
                    // the next batch's logits beside this one's values: the exchanges wait on
                    // shuffles that the values' arithmetic hides
                    f = over_g((uint32_t)jr);
                    angles(f, cs, sn);
                    float y = logit(0, false);
#pragma unroll 1
                    for (int kk = 0; kk < C::RUN - KB; kk += KB) {
                        const float w = weight(y, kk);
                        y = logit(kk + KB, false);
                        values(w, kk, false);
                    }
                    values(weight(y, C::RUN - KB), C::RUN - KB, false);
                } else {
#pragma unroll 1
                    for (int kk = 0; kk < C::RUN; kk += KB) values(weight(logit(kk, true), kk), kk, true);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
            }
            i += cnt;
            e += cnt;
        }
        // the warp's groups joined, then the key groups through shared memory
        float top = ref;
#pragma unroll
        for (int w = LPK; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        const float scale = ref == -INFINITY ? 0.f : exp2f(ref - top);
        l *= scale;
#pragma unroll
        for (int w = R; w < 32; w <<= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
        if (lane < R) ml[warp * R + lane] = make_float2(top, l);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float a = __shfl_sync(0xffffffffu, scale, r, LPK);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                o[r][u] = a == 0.f ? make_float2(0.f, 0.f) : mul2(o[r][u], make_float2(a, a));
#pragma unroll
                for (int w = LPK; w < 32; w <<= 1) {
                    o[r][u].x += __shfl_xor_sync(0xffffffffu, o[r][u].x, w);
                    o[r][u].y += __shfl_xor_sync(0xffffffffu, o[r][u].y, w);
                }
            }
            if (grp == 0) {
                float* to = red + (warp * R + r) * D + m0;
                *reinterpret_cast<float4*>(to) = make_float4(o[r][0].x, o[r][0].y, o[r][1].x, o[r][1].y);
                *reinterpret_cast<float4*>(to + H) = make_float4(o[r][2].x, o[r][2].y, o[r][3].x, o[r][3].y);
            }
        }
        if (named_or(!ok)) return;
        const bool whole = walk.i0 == 0 && walk.i1 == s.items;
        if (tid == 0 && walk.i0 == 0 && !whole) note_cut(p, s, plan->per, walk.cur, walk.kvh, walk.r0, nrows);
        float* part = reinterpret_cast<float*>(p.workspace + kPagedHeader) +
                      ((size_t)blockIdx.x * 2 + (walk.i0 == 0 ? 1 : 0)) * RT * (D + 4);
        for (int x = tid; x < nrows * (D / 4); x += CT) {
            const int r = x / (D / 4), c = x % (D / 4) * 4, w0 = r / R;  // warps w0, w0 + WR, ... hold the row
            float M = -INFINITY;
#pragma unroll
            for (int k = 0; k < C::WK; ++k) M = fmaxf(M, ml[(k * C::WR + w0) * R + r % R].x);
            const float base = M == -INFINITY ? 0.f : M;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < C::WK; ++k) {
                const int y = (k * C::WR + w0) * R + r % R;
                const float2 t = ml[y];
                if (t.x == -INFINITY && t.y == 0.f) continue;  // no key of this row
                const float f = exp2f(t.x - base);
                const float4 v = *reinterpret_cast<const float4*>(red + y * D + c);
                a.x = fmaf(f, v.x, a.x);
                a.y = fmaf(f, v.y, a.y);
                a.z = fmaf(f, v.z, a.z);
                a.w = fmaf(f, v.w, a.w);
                sum = fmaf(f, t.y, sum);
            }
            if (whole) {
                const int node = (walk.r0 + r) / p.group, hd = walk.kvh * p.group + (walk.r0 + r) % p.group;
                float* out = static_cast<float*>(p.out) + ((size_t)(s.n0 + node) * p.Hq + hd) * D + c;
                *reinterpret_cast<float4*>(out) = make_float4(a.x / sum, a.y / sum, a.z / sum, a.w / sum);
            } else {
                *reinterpret_cast<float4*>(part + (size_t)r * (D + 4) + c) = a;
                if (c == 0) *reinterpret_cast<float2*>(part + (size_t)r * (D + 4) + D) = make_float2(M, sum);
            }
        }
        walk.done();
    }
}

template <int D, int RT>
cudaError_t run(const PagedProblem& p, cudaStream_t st, int* grid)
{
    constexpr int smem = Cfg<D, RT>::END;
    static PerDevice once;
    int nsm = 0;
    cudaError_t e = once.get(&nsm, [](int* n, int dev) {
        cudaError_t err = cudaFuncSetAttribute(decode_paged_fp32_kernel<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        cudaFuncAttributes a;
        if (err == cudaSuccess) err = cudaFuncGetAttributes(&a, decode_paged_fp32_kernel<D, RT>);
        // fewer registers at launch would leave setmaxnreg waiting
        if (err == cudaSuccess && a.numRegs * NTHR < (2 * R_CALC + R_PROD) * 128) err = cudaErrorInvalidKernelImage;
        return err == cudaSuccess ? cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev) : err;
    });
    if (e != cudaSuccess) return e;
    *grid = std::min(nsm, kCtas);
    decode_paged_fp32_kernel<D, RT><<<*grid, NTHR, smem, st>>>(p, p.wait_cycles > 0 ? p.wait_cycles : kWaitCycles);
    return cudaGetLastError();
}

template <int D>
cudaError_t run_rows(const PagedProblem& p, int rt, cudaStream_t st, int* grid)
{
    switch (rt) {
        case 4: return run<D, 4>(p, st, grid);
        case 8: return run<D, 8>(p, st, grid);
        case 16: return run<D, 16>(p, st, grid);
        default: return run<D, 32>(p, st, grid);
    }
}

}  // namespace

// rows of a unit for `rows` query rows per request and kv head
int paged_fp32_rows(int rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }
size_t paged_fp32_workspace(int rows, int d) { return (size_t)kCtas * 2 * paged_fp32_rows(rows) * (d + 4) * sizeof(float); }

cudaError_t launch_decode_paged_fp32(const PagedProblem& p, int d, cudaStream_t s, int* grid)
{
    const int rt = paged_fp32_rows(p.max_nodes * p.group);
    return d == 64 ? run_rows<64>(p, rt, s, grid) : run_rows<128>(p, rt, s, grid);
}

}  // namespace jl
