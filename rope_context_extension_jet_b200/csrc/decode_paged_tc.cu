// decode_paged_tc.cu -- bf16 decode over a paged raw-key cache on the tensor
// cores: one new row or a tree of drafted rows per request (mathematics and
// work plan: decode_paged.cu, paged_common.cuh).
//
// A unit is (request, kv head, up to RT query rows); its keys come in tiles of
// 128.  Per tile, with the keys as the 128 rows of the first product so that its
// cost follows the number of query rows:
//   S^T [128 keys x RT]  = K_rot [128 x d] Q_rot^T [d x RT]   (fp16 operands)
//   O^T [d x RT]        += V^T [d x 128] P^T [128 x RT]       (bf16 operands; P as two
//                          terms, for which a product of 64 columns has room)
// both accumulated in fp32 in tensor memory.  A softmax thread owns one key (one
// TMEM lane) and walks the RT columns, so the weights of a key leave as whole
// 16-byte chunks; each thread sums its own key's weights.  The running
// maximum of a column only has to be near: weights are fp32 / bf16, whose range is
// far wider than the 2^40 that logits may rise by before it is taken again (kAbove),
// so each tile costs one vote of the 128 threads, and only a tile that passes the
// reference takes exact column maxima and rescales O and the sums.
//
// Warp roles:
//   warp 0      K producer: page numbers of a tile's rows, one TMA box per page
//   warp 3      V producer
//   warp 1      MMA issuer
//   warp 2      TMEM allocation; planner: the piece's units, a few ahead, for the others
//   warps 4-11  per unit: the tree, positions, query scales; per phase: the rotated
//               queries; per tile: keys rotated in shared memory, in place (angles
//               advance from row to row)
//   warps 12-.. softmax, one warpgroup per NCOL columns
// Every wait on a barrier is bounded as in the prefill kernels.
//
// Bound: HBM at 128K (8 requests, 32 query heads on 8, d = 128: 649-660 us one call right
// after another, 6.5 TB/s of K and V, 800 where every call has another cache); the
// rotation of the key tiles where there are more rows or phases (8 x 32K: 4 nodes 189 us,
// 8 nodes 242 us; bytes alone 162 us).
#include <algorithm>

#include "paged_tc_roles.cuh"

namespace jl {
namespace ptc {
namespace {

template <int D, int NCOL>
struct CfgTiles {
    static constexpr int DIM = D, ROWS = NCOL;
    static constexpr int NSK = D == 64 ? 6 : 3, NSV = D == 64 ? 4 : 2;  // 16 / 32 KB stages
    // columns of the second product (one swizzle atom is 64 wide): the weights' upper
    // bits from 0 on, the rest of them from 32 on
    static constexpr int NPV = 64, REST = 32;
    static constexpr int NP = 2;        // P buffers
    static constexpr int THREADS = 512;
    // the two rotation warpgroups take tiles in turn (one's latencies under the
    // other's arithmetic)
    static constexpr bool ALT = true;
    static constexpr int ROT = 128, ROTALL = 256, SOFT = 4;
    static constexpr int ATOMS = D / 64;
    static constexpr int TILE = KT * D * 2, ATOM_K = KT * 128, ATOM_Q = NCOL * 128;
    static constexpr int K0 = 0, V0 = K0 + NSK * TILE, P0 = V0 + NSV * TILE, PBYTES = KT * NPV * 2;
    static constexpr int Q0 = P0 + NP * PBYTES, QBYTES = NCOL * D * 2;
    static constexpr int BASE = Q0 + (QBYTES + 1023) / 1024 * 1024;
    static __device__ __forceinline__ uint32_t q_off(int r, int ch) { return tc::sw128_off<NCOL>(r, ch); }
};
template <int D, int NCOL>
struct Cfg : CfgTiles<D, NCOL>,
             Notes<D, NCOL, CfgTiles<D, NCOL>::NSK, CfgTiles<D, NCOL>::NSV, CfgTiles<D, NCOL>::BASE, 6, 16> {
    static constexpr int M0 = Cfg::NOTES_END;               // [NCOL] minus the column references, [NCOL] zeros, [NCOL] ones
    static constexpr int RED = M0 + NCOL * 12;              // [4][NCOL] column maxima / sums, [NCOL] rescale factors
    static constexpr int TOTAL = RED + 5 * NCOL * 4 + 1024;
    static_assert(TOTAL <= 232448, "shared memory");
};

// Transposing reduction over a warp of 16 columns: lanes l and l + 16 return op
// over the 32 lanes of v[l] (v is consumed).
template <bool MAX>
__device__ __forceinline__ float lane_columns(float (&v)[16], int lane)
{
#pragma unroll
    for (int w = 8; w >= 1; w >>= 1) {
        const bool hi = lane & w;
#pragma unroll
        for (int x = 0; x < w; ++x) {
            const float give = hi ? v[x] : v[x + w], keep = hi ? v[x + w] : v[x];
            const float got = __shfl_xor_sync(0xffffffffu, give, w);
            v[x] = MAX ? fmaxf(keep, got) : keep + got;
        }
    }
    const float got = __shfl_xor_sync(0xffffffffu, v[0], 16);
    return MAX ? fmaxf(v[0], got) : v[0] + got;
}

template <int D, int NCOL>
__global__ void __launch_bounds__(Cfg<D, NCOL>::THREADS, 1)
    decode_paged_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                           const __grid_constant__ PagedProblem p, const Launch ln)
{
    using C = Cfg<D, NCOL>;
    constexpr int NSK = C::NSK, NSV = C::NSV;
    unsigned char* const smem = smem_base();
    const Role<C> ro(p, ln);
    const Bars<C> bars;
    uint64_t *sfull = bars.extra, *pfull = sfull + 2, *pvdone = pfull + 2;
    const int warp = ro.warp, lane = ro.lane;
    constexpr uint32_t TCOLS = 256, TS = C::NPV;  // S at 0 and TS, O at 2 TS
    const uint32_t tmem = start_cta<C, TCOLS>(ro, [&] {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sfull[s], 1);
            mbar_init(&pfull[s], 4);
            mbar_init(&pvdone[s], 1);
        }
    });
    if (warp == 0) {
        produce<C, true>(ro, &tmK);
    } else if (warp == 3) {
        produce<C, false>(ro, &tmV);
    } else if (warp == 2) {
        plan_units<C>(ro);
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        constexpr uint32_t IQK = idesc_f16(KT, NCOL, 0);
        constexpr uint32_t IPV = idesc_bf16(128, C::NPV, 1) | (1u << 15);  // A (V^T) and B (P^T) both MN-major
        const uint32_t sb = smem_u32(smem);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        int e = 0;
        unsigned nfix = 0;  // per stage: parity of the repaired value tiles so far
        bool ok = true;
        // O^T += V^T P^T of item x
        auto pv = [&](int x, bool first, bool fix) {
            if (!ro.wait(&pfull[x & 1], (x >> 1) & 1, 0x611)) return false;
            const int st = x % NSV;
            if (!ro.wait(&bars.vfull[st], (x / NSV) & 1, 0x612)) return false;
            if (fix) {
                if (!ro.wait(&bars.vfix[st], (nfix >> st) & 1, 0x613)) return false;
                nfix ^= 1u << st;
            }
            tc_fence_after();
            // d = 64: the second 64-column atom of V^T is whatever follows the tile; it
            // fills lanes 64..127 of O^T, which nothing reads
            umma_ss_mn128(tm + 2 * TS, sdesc_sw128(sb + C::V0 + st * C::TILE, C::ATOM_K, 1024),
                          sdesc_sw128(sb + C::P0 + (x % C::NP) * C::PBYTES, C::ATOM_K, 1024), IPV, first ? 0u : 1u);
            umma_commit_elect(&bars.vempty[st]);
            umma_commit_elect(&pvdone[x & 1]);
            return true;
        };
        bool pend = false, pfirst = false, pfix = false;
        int phases = 0;
        const unsigned all_pages = ro.all_pages();
        for (int k = 0; ok; ++k) {
            if (!ro.unit_wait(k, 0x616)) { ok = false; break; }
            UnitPtr un = ro.unit(k);
            if (un->rows == 0) break;
            const int L = un->L;
            int gcur = -1;
            bool first = true;
            for (UnitItems it(un); it.left > 0; it.next(), ++e) {
                const int st = e % NSK;
                if (it.g != gcur) {
                    gcur = it.g;
                    if (!ro.wait(bars.qready, phases & 1, 0x615)) { ok = false; break; }
                    ++phases;
                }
                if (!ro.wait(&bars.kready[st], (e / NSK) & 1, 0x614)) { ok = false; break; }
                const bool fix = (it.tile + 1) * KT > L || ro.note()[e % INFO] != all_pages;
                tc_fence_after();
                const uint64_t a = sdesc_sw128(sb + C::K0 + st * C::TILE, 16, 1024);
                const uint64_t bq = sdesc_sw128(sb + C::Q0, 16, 1024);
                umma_ss_k64(tm + (e & 1) * TS, a, bq, IQK, 0u);
                if (D == 128) umma_ss_k64(tm + (e & 1) * TS, a + C::ATOM_K / 16, bq + C::ATOM_Q / 16, IQK, 1u);
                umma_commit_elect(&bars.kempty[st]);
                umma_commit_elect(&sfull[e & 1]);
                if (pend && !pv(e - 1, pfirst, pfix)) { ok = false; break; }
                pend = true;
                pfirst = first;
                pfix = fix;
                first = false;
            }
            ro.unit_done(k);
        }
        if (ok && pend) pv(e - 1, pfirst, pfix);
        umma_commit_elect(bars.drain);
        mbar_wait(bars.drain, 0);
    } else if (warp < 12) {
        rotate_keys<C>(ro);
    } else {
        // ------------------------------------------------------ softmax
        constexpr int bid = 2;  // named barrier of the warpgroup
        const int wl = warp & 3, key = wl * 32 + lane;
        const float* ksc = reinterpret_cast<const float*>(smem + C::KSC);
        const uint32_t tl = tmem + ((uint32_t)(32 * wl) << 16);
        float* nref = reinterpret_cast<float*>(smem + C::M0);
        float *zero = nref + NCOL, *one = zero + NCOL;
        float* red = reinterpret_cast<float*>(smem + C::RED);
        float* alpha = red + 4 * NCOL;
        float l[NCOL];  // sums over this thread's keys
        int e = 0, nu = 0;
        // as above, a wait that ran out is carried to the warpgroup's next barrier,
        // where its four warps stop together
        bool ok = true, stop = false;
        const int gshift = min(p.page_shift, 7);
        const unsigned all_pages = ro.all_pages();
        for (; !stop; ++nu) {
            ok = ro.unit_wait(nu, 0x636);
            UnitPtr ud = ro.unit(nu);
            if (ok && ud->rows == 0) {
                named_or(bid, 128, false);  // meets a warp that gave up waiting for the unit
                break;
            }
            const unsigned char* un = smem + C::UNIT + (nu & 1) * C::UBYTES;
            const int* depth = reinterpret_cast<const int*>(un + C::U_DEPTH);
            const int* clim = reinterpret_cast<const int*>(un + C::U_LIM);
            const int* qG = reinterpret_cast<const int*>(un + C::U_QG);
            const float* cq = reinterpret_cast<const float*>(un + C::U_CQ);
            const unsigned long long* canc = reinterpret_cast<const unsigned long long*>(un + C::U_ANC);
            ok = ok && ro.wait(&bars.uready[nu & 1], (nu >> 1) & 1, 0x631);
#pragma unroll
            for (int c = 0; c < NCOL; ++c) l[c] = 0.f;
            if (key < NCOL) {
                nref[key] = key < ud->rows ? -kNoRef : 0.f;  // (a column without a query is no reason to move one)
                zero[key] = 0.f;
                one[key] = 1.f;
            }
            if (named_or(bid, 128, !ok)) break;
            const int cols = ud->rows, L = ud->L, n = L + ud->T;
            // an exact item has pairs of the other branch up to tile edge `near`, a remote
            // one past `far` (always, where group sizes differ)
            const int near = n - 1 - ud->w0;
            const int far = ud->ng > 1 ? -1 : (int)max(-1ll, (long long)L - ud->w0 - (KT - 1));
            bool first = true;
            for (UnitItems it(ud); it.left > 0; it.next(), ++e) {
                const int g = it.g, j0 = it.tile * KT;
                ok = ok && ro.wait(&sfull[e & 1], (e >> 1) & 1, 0x632);
                tc_fence_after();
                const unsigned have = ro.note()[e % INFO];
                // which pairs of the tile this item leaves out: some of a drafted or
                // incomplete tile's; the other branch's on the border of the window
                // (or of columns with another group size)
                const bool drafted = j0 + KT > L || have != all_pages;
                const bool masked = drafted || (g == 0 ? j0 <= near : j0 > far);
                // rotation warp wl scaled some of this warp's key rows
                const bool any_scaled = reinterpret_cast<const volatile unsigned*>(smem + C::SCALED)[(e % INFO) * 8 + wl] != 0;
                float ks = 1.f;
                if (any_scaled) ks = *reinterpret_cast<const volatile float*>(ksc + (e % INFO) * KT + key);
                const int j = j0 + key, u = j - L;
                const bool there = j < n && ((have >> (key >> gshift)) & 1);
                uint32_t keep = 0;  // masked tiles: one bit per column
                if (masked) {
                    asm volatile("" ::: "memory");  // a branch, not predication: most tiles skip this
                    const int kpos = there ? (u < 0 ? j : L + depth[u]) : 0;
                    const unsigned long long self = u < 0 ? ~0ull : 1ull << (u & 63);
#pragma unroll 4
                    for (int c = 0; c < NCOL; ++c) {
                        const bool local = kpos > clim[c];
                        const bool mine = g == 0 ? local : (!local && qG[c] == g);
                        keep |= (uint32_t)(mine && there && (u < 0 || (canc[c] & self))) << c;
                    }
                }
                // logits in log2 units, plus nm (minus their references, or
                // nothing); what this item leaves out is -inf
                auto logits = [&](float (&y)[NCOL], const float* nm) {
                    {
                        uint32_t raw[NCOL];
#pragma unroll
                        for (int c = 0; c < NCOL; c += 16)
                            if (c < cols) tmem_ld16(tl + (e & 1) * TS + c, raw + c);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < NCOL; ++c) y[c] = __uint_as_float(raw[c]);
                    }
                    if (any_scaled) {  // the whole factor here, 1 below
                        asm volatile("" ::: "memory");
#pragma unroll
                        for (int c = 0; c < NCOL; ++c) y[c] *= logit_factor(cq[c], ks);
                    }
                    const float* factor = any_scaled ? one : cq;
#pragma unroll
                    for (int cb = 0; cb < NCOL; cb += 16) {
                        if (cb < cols) {
                            asm volatile("" ::: "memory");  // scales of 16 columns at a time: registers
#pragma unroll
                            for (int c = cb; c < cb + 16; c += 4) {
                                const float4 k4 = *reinterpret_cast<const float4*>(factor + c);
                                const float4 m4 = *reinterpret_cast<const float4*>(nm + c);
                                const float2 a = fma2(make_float2(y[c], y[c + 1]), make_float2(k4.x, k4.y), make_float2(m4.x, m4.y));
                                const float2 b = fma2(make_float2(y[c + 2], y[c + 3]), make_float2(k4.z, k4.w), make_float2(m4.z, m4.w));
                                y[c] = a.x;
                                y[c + 1] = a.y;
                                y[c + 2] = b.x;
                                y[c + 3] = b.y;
                            }
                        }
                    }
                    if (masked) {
                        asm volatile("" ::: "memory");
                        const uint32_t bits = keep;
#pragma unroll
                        for (int c = 0; c < NCOL; ++c) y[c] = (bits >> c) & 1 ? y[c] : -INFINITY;
                    }
                };
                float y[NCOL];
                for (bool rel = !first;; rel = !rel) {  // the first tile sets its references first
                    float top = -INFINITY;
                    {
                        logits(y, rel ? nref : zero);
                        if (rel) {
#pragma unroll
                            for (int c = 0; c < NCOL; c += 2)
                                if ((c & ~15) < cols) top = fmax3(top, y[c], y[c + 1]);
                        } else {
                            // exact column maxima over this warp's keys
#pragma unroll
                            for (int cb = 0; cb < NCOL; cb += 16) {
                                if (cb >= cols) break;
                                float v[16];
#pragma unroll
                                for (int c = 0; c < 16; ++c) v[c] = y[cb + c];
                                const float m = lane_columns<true>(v, lane);
                                if (lane < 16) red[wl * NCOL + cb + lane] = m;
                            }
                        }
                    }
                    if (rel) {
                        if (!named_or(bid, 128, top > kExceed || !ok)) break;
                        if (named_or(bid, 128, !ok)) {
                            stop = true;
                            break;
                        }
                        continue;
                    }
                    // sums and O follow the new references
                    named_sync(bid, 128);
                    if (key < NCOL && key < (cols + 15) / 16 * 16) {
                        const float m = fmaxf(fmaxf(red[key], red[NCOL + key]), fmaxf(red[2 * NCOL + key], red[3 * NCOL + key]));
                        const float old = -nref[key];
                        float a = 1.f;
                        if (m > -INFINITY && m + kAbove > old) {
                            nref[key] = -(m + kAbove);
                            a = exp2f(old - (m + kAbove));
                        }
                        alpha[key] = a;
                    }
                    named_sync(bid, 128);
#pragma unroll
                    for (int c = 0; c < NCOL; ++c)
                        if ((c & ~15) < cols) l[c] *= alpha[c];
                    if (!first) {
                        ok = ro.wait(&pvdone[(e - 1) & 1], ((e - 1) >> 1) & 1, 0x633);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < NCOL; c += 16) {
                            if (c >= cols) break;
                            uint32_t o[16];
#pragma unroll 1
                            for (int at = c; at < C::NPV; at += C::REST) {
                                tmem_ld16(tl + 2 * TS + at, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha[c + x]);
                                tmem_st16(tl + 2 * TS + at, o);
                            }
                        }
                        tmem_wait_st();
                    }
                    if (named_or(bid, 128, !ok)) {  // and alpha is read before it is written again
                        stop = true;
                        break;
                    }
                }
                if (stop) break;
                first = false;
                // weights to the P buffer e % 2: P V of item e - 2, its last reader, was issued
                // before Q K^T of this item, whose commit (sfull) covers every earlier MMA
                static_assert(C::NP == 2, "P buffers");
                unsigned char* pb = smem + C::P0 + (e % C::NP) * C::PBYTES + key * 128;
                {
#pragma unroll
                    for (int c = 0; c < NCOL; c += 8) {
                        if ((c & ~15) < cols) {
                            uint32_t o[4], rest[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const float a = ex2_approx(y[c + 2 * x]), b = ex2_approx(y[c + 2 * x + 1]);
                                l[c + 2 * x] += a;
                                l[c + 2 * x + 1] += b;
                                o[x] = split_weights(a, b, rest[x]);
                            }
                            *reinterpret_cast<uint4*>(pb + (((c >> 3) ^ (key & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<uint4*>(pb + ((((c + C::REST) >> 3) ^ (key & 7)) << 4)) =
                                make_uint4(rest[0], rest[1], rest[2], rest[3]);
                        }
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[e & 1]);
            }
            if (stop) break;
            // ---- the unit's piece is complete
            ok = ok && ro.wait(&pvdone[(e - 1) & 1], ((e - 1) >> 1) & 1, 0x635);
            tc_fence_after();
#pragma unroll
            for (int cb = 0; cb < NCOL; cb += 16) {
                float v[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) v[c] = l[cb + c];
                const float sum = lane_columns<false>(v, lane);
                if (lane < 16) red[wl * NCOL + cb + lane] = sum;
            }
            if (named_or(bid, 128, !ok)) break;
            const int i0 = ud->i0, r0 = ud->r0, kvh = ud->kvh, n0 = ud->n0;
            const bool whole = i0 == 0 && ud->i1 == ud->items;
            const unsigned long long bad = ud->bad;
            float* part = reinterpret_cast<float*>(p.workspace + kPagedHeader) +
                          ((size_t)blockIdx.x * 2 + (i0 == 0 ? 1 : 0)) * NCOL * (D + 4);
            // lane c looks after column c: its sum and where its row goes
            const int node0 = r0 / p.group, mine = min(lane, cols - 1);
            const float sum = red[mine] + red[NCOL + mine] + red[2 * NCOL + mine] + red[3 * NCOL + mine];
            const float inv = whole ? __fdividef(1.f, sum) : 1.f;
            const int to = whole ? ((r0 + mine) / p.group - node0) * p.Hq + (r0 + mine) % p.group : mine;
            __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.out) + ((size_t)(n0 + node0) * p.Hq + kvh * p.group) * D + key;
            if (!whole && wl == 0 && lane < cols)
                *reinterpret_cast<float2*>(part + lane * (D + 4) + D) =
                    make_float2(nref[lane] == -kNoRef ? -INFINITY : -nref[lane], sum);
#pragma unroll
            for (int cb = 0; cb < NCOL; cb += 16) {
                if (cb >= cols) break;
                uint32_t o[16], rest[16];
                tmem_ld16(tl + 2 * TS + cb, o);
                tmem_ld16(tl + 2 * TS + C::REST + cb, rest);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const int row = __shfl_sync(0xffffffffu, to, cb + x);
                    const float val = (__uint_as_float(o[x]) + __uint_as_float(rest[x])) * __shfl_sync(0xffffffffu, inv, cb + x);
                    if (key < D && cb + x < cols) {
                        if (whole)
                            orow[(size_t)row * D] = __float2bfloat16_rn(val);
                        else
                            part[row * (D + 4) + key] = val;
                    }
                }
            }
            if (bad && key < D) {
                // infinities and NaN of drafted rows a node attends: they outweigh what this
                // thread has just written
                for (int c = 0; c < cols; ++c) {
                    for (unsigned long long rest = bad & canc[c]; rest; rest &= rest - 1) {
                        const int row = L + __ffsll((long long)rest) - 1;
                        const int page = p.table[(size_t)ud->b * p.max_pages + (row >> p.page_shift)];
                        const float v = __bfloat162float(static_cast<const __nv_bfloat16*>(p.vc)[
                            (((size_t)page * p.Hkv + kvh) * p.page_size + (row & (p.page_size - 1))) * D + key]);
                        if (fabsf(v) < INFINITY) continue;
                        const int node = (r0 + c) / p.group - node0, hd = (r0 + c) % p.group;
                        __nv_bfloat16* x = orow + (size_t)(node * p.Hq + hd) * D;
                        if (whole)
                            *x = __float2bfloat16_rn(__bfloat162float(*x) + v);
                        else
                            part[c * (D + 4) + key] += v;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.ufree[nu & 1]);
            named_sync(bid, 128);  // red and nref are read before the next unit writes them
            ro.unit_done(nu);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, TCOLS);
    }
}

template <int D, int NCOL>
cudaError_t run(const PagedProblem& p, const Launch& ln, cudaStream_t st, int* grid)
{
    CUtensorMap tk, tv;
    cudaError_t e;
    const int planes = p.num_pages * p.Hkv, box = std::min(p.page_size, KT);
    if ((e = tc::make_map(&tk, p.kc, D, p.page_size, p.page_size, planes, box)) != cudaSuccess) return e;
    if ((e = tc::make_map(&tv, p.vc, D, p.page_size, p.page_size, planes, box)) != cudaSuccess) return e;
    constexpr int smem = Cfg<D, NCOL>::TOTAL;
    auto kern = decode_paged_tc_kernel<D, NCOL>;
    static PerDevice once;
    int nsm = 0;
    e = once.get(&nsm, [&](int* n, int dev) {
        cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        return err == cudaSuccess ? cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev) : err;
    });
    if (e != cudaSuccess) return e;
    *grid = std::min(nsm, kTcCtas);
    kern<<<*grid, Cfg<D, NCOL>::THREADS, smem, st>>>(tk, tv, p, ln);
    return cudaGetLastError();
}

}  // namespace

cudaError_t run_cols(const PagedProblem& p, int d, int cols, const Launch& ln, cudaStream_t st, int* grid)
{
    if (d == 64) return cols <= 16 ? run<64, 16>(p, ln, st, grid) : run<64, 32>(p, ln, st, grid);
    return cols <= 16 ? run<128, 16>(p, ln, st, grid) : run<128, 32>(p, ln, st, grid);
}

}  // namespace ptc
}  // namespace jl
