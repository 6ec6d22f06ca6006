// decode_paged_rows.cu -- bf16 decode over a paged raw-key cache for more than 32
// query rows per request and kv head (larger drafted trees, wide head groups), with
// the query rows as the 128 rows of the products (mathematics and work plan:
// decode_paged.cu, paged_common.cuh; shared roles: paged_tc_roles.cuh).
//
//   S [128 rows x 128 keys] = Q_rot [128 x d] K_rot^T      (fp16 operands)
//   O [128 rows x d]       += P [128 x 128] V              (bf16 operands, P in TMEM; for
//                                                           half of the keys as two terms)
// A softmax thread owns half of a row (64 keys of one TMEM lane), so the running
// reference, the sum and the rescale factor are its own and no element needs a
// per-column factor; from about 32 rows on that beats the form of decode_paged_tc.cu,
// whose cost per key grows with the rows.  Two "streams" (S, O) overlap: the softmax
// warps take them in turn, all eight on one, while the tensor cores work for the
// other.  (With one warpgroup per stream a thread held the whole row and had to read
// half of it from tensor memory twice: 64-node trees at 8 x 32K 404 us instead of 372.)
//   ROWS = 256: stream s holds rows [128 s, 128 s + 128); both use every key tile,
//     which is loaded and rotated once for all 256.
//   ROWS = 128: both hold the same rows and take the tiles in turn; each keeps its
//     own reference, sum and O, joined where the unit ends.
//
// Warp roles: 0 / 3 producers, 1 MMA issuer, 2 tensor memory and planner, 4-11
// rotation, 12-15 / 16-19 softmax of the first / second 64 keys of a tile.
// TMEM (512 columns): S_0, S_1 (128 each; P_s over S_s, each half over the half it was
// made from: the weights in columns 0-31, what they leave of 16 bits in 32-47), O_0,
// O_1.
//
// Bound: latencies in the softmax (8 x 32K rows: 16 nodes 261 us, 64 nodes 471 us; 64
// nodes at 8 x 128K 1.72-1.87 ms, where bytes and products each take 0.66 ms).  A tile of
// 256 rows takes about 5500 cycles, of which the exponentials need 2048 and the products
// 2560, with half of the issue slots empty: a thread loads all of its 64 scores before
// the first exponential, and the wait for S and the agreement of the two warps that
// share rows stand beside that.  Exponentials on the FMA pipes made it slower (an eighth
// of them 6%).
#include <algorithm>

#include "paged_tc_roles.cuh"

namespace jl {
namespace ptc {
namespace {

template <int D, int NROWS>
struct RowTiles {
    static constexpr int DIM = D, ROWS = NROWS;
    static constexpr int NSK = D == 64 ? 4 : NROWS == 128 ? 3 : 2, NSV = D == 64 ? 4 : 2;
    static constexpr int THREADS = 640;
    // two rotation warpgroups: in turn where the ring has three key stages, else
    // sharing each tile.  (One alone took 4200 cycles a tile and bounded the kernel.)
    static constexpr bool ALT = NSK >= 3;
    static constexpr int ROT = ALT ? 128 : 256, ROTALL = 256, SOFT = 8;
    static constexpr int ATOMS = D / 64;
    static constexpr int TILE = KT * D * 2, ATOM_K = KT * 128;
    static constexpr int K0 = 0, V0 = K0 + NSK * TILE, Q0 = V0 + NSV * TILE, BASE = Q0 + NROWS * D * 2;
    static __device__ __forceinline__ uint32_t q_off(int r, int ch) { return (r >> 7) * TILE + tc::sw128_off<128>(r & 127, ch); }
};
template <int D, int NROWS>
struct RowCfg : RowTiles<D, NROWS>,
                Notes<D, NROWS, RowTiles<D, NROWS>::NSK, RowTiles<D, NROWS>::NSV, RowTiles<D, NROWS>::BASE, 6, 20> {
    static constexpr int XCH = RowCfg::NOTES_END;  // [2][128] sums of both streams over a half's keys
    static constexpr int TOP = XCH + 2 * 128 * 8;  // [2][2][128] largest logit of a half's keys, per stream
    static constexpr int TOTAL = TOP + 2 * 2 * 128 * 4 + 1024;
    static_assert(TOTAL <= 232448, "shared memory");
    // Registers per thread after setmaxnreg: producers / issuer / planner, the two
    // rotation and the two softmax warpgroups.  640 threads launch with 96 each, and an
    // increase draws on that.
    static constexpr int R_PROD = 40, R_ROT = 88, R_SOFT = 128;
    static_assert((R_PROD + 2 * R_ROT + 2 * R_SOFT) * 128 <= 640 * 96, "register split");
};

template <int D, int NROWS>
__global__ void __launch_bounds__(640, 1)
    decode_paged_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                             const __grid_constant__ PagedProblem p, const Launch ln)
{
    using C = RowCfg<D, NROWS>;
    constexpr bool PAIR = NROWS == 256;
    // 32-key parts of a half whose weights keep 16 bits (split_weights): here, unlike in
    // decode_paged_tc.cu, each costs a product and the softmax's time.  128K trees of 64
    // nodes, with the row maximum still taken on every tile: error 2.4e-3 (rms, of the
    // results) and 1779 us with none, 2.2e-3 and 1939 us with one of the two, 1.9e-3 and
    // 2238 us with both; rounding the results alone is 1.6e-3.  (So a row is less exact
    // here than in decode_paged_tc.cu, which keeps both terms.)
    constexpr int PARTS = 1;
    constexpr float kSumMax = 65536.f;  // 2^kExceed
    static_assert(kExceed == 16.f && PARTS == 1, "weights");
    constexpr int NSK = C::NSK, NSV = C::NSV;
    unsigned char* const smem = smem_base();
    const Role<C> ro(p, ln);
    const Bars<C> bars;
    uint64_t *sfull = bars.extra, *pfull = sfull + 2, *pvdone = pfull + 2;  // per stream
    const int warp = ro.warp, lane = ro.lane;
    const uint32_t tmem = start_cta<C, 512>(ro, [&] {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sfull[s], 1);
            mbar_init(&pfull[s], C::SOFT);
            mbar_init(&pvdone[s], 1);
        }
    });
    if (warp < 4) {
        regs_dec<C::R_PROD>();
        if (warp == 0) {
            produce<C, true>(ro, &tmK);
        } else if (warp == 3) {
            produce<C, false>(ro, &tmV);
        } else if (warp == 2) {
            plan_units<C>(ro);
        } else {
            // -------------------------------------------------- MMA issuer
            // A task is one item on one stream: S_s = Q K^T, later O_s += P_s V.  P_s
            // lies over S_s, so a stream's P V is issued before its next Q K^T (one
            // issuer's MMAs run in order).
            constexpr uint32_t IQK = idesc_f16(128, KT, 0), IPV = idesc_bf16(128, D, 1);
            const uint32_t sb = smem_u32(smem);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            int e = 0, phases = 0;
            unsigned nfix = 0;              // per stage: parity of the repaired value tiles so far
            int done[2] = {0, 0};           // P V of each stream so far
            int pe[2] = {-1, -1};           // its pending item
            bool pfirst[2] = {false, false}, pfix[2] = {false, false};
            bool ok = true;
            const unsigned all_pages = ro.all_pages();
            auto pv = [&](int s) {
                const int x = pe[s], st = x % NSV;
                if (!ro.wait(&bars.vfull[st], (x / NSV) & 1, 0x512)) return false;
                if (pfix[s] && !(PAIR && s == 1)) {  // both streams use the tile: stream 0 comes first
                    if (!ro.wait(&bars.vfix[st], (nfix >> st) & 1, 0x513)) return false;
                    nfix ^= 1u << st;
                }
                if (!ro.wait(&pfull[s], done[s] & 1, 0x511)) return false;
                tc_fence_after();
                const uint64_t vd = sdesc_sw128(sb + C::V0 + st * C::TILE, C::ATOM_K, 1024);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    umma_pv_k64(tm + 256 + s * 128, tm + s * 128 + 64 * half, vd + 512 * half, IPV, pfirst[s] && half == 0 ? 0u : 1u);
                    for (int part = 0; part < PARTS; ++part)
                        umma_ts_k32(tm + 256 + s * 128, tm + s * 128 + 64 * half + 32 + 16 * part, vd + 512 * half + 256 * part, IPV);
                }
                umma_commit_elect(&pvdone[s]);
                if (!PAIR || s == 1) umma_commit_elect(&bars.vempty[st]);
                ++done[s];
                pe[s] = -1;
                return true;
            };
            for (int k = 0; ok; ++k) {
                if (!ro.unit_wait(k, 0x516)) break;
                UnitPtr un = ro.unit(k);
                if (un->rows == 0) break;
                const int L = un->L;
                int gcur = -1, li = 0;
                for (UnitItems it(un); ok && it.left > 0; it.next(), ++e, ++li) {
                    const int st = e % NSK;
                    bool fix = false;
                    for (int s = PAIR ? 0 : li & 1, s1 = PAIR ? 1 : s; s <= s1; ++s) {
                        if (pe[s] >= 0 && !pv(s)) { ok = false; break; }
                        if (s == 0 || !PAIR) {
                            if (it.g != gcur) {
                                gcur = it.g;
                                if (!ro.wait(bars.qready, phases & 1, 0x515)) { ok = false; break; }
                                ++phases;
                            }
                            if (!ro.wait(&bars.kready[st], (e / NSK) & 1, 0x514)) { ok = false; break; }
                            fix = (it.tile + 1) * KT > L || ro.note()[e % INFO] != all_pages;
                        }
                        tc_fence_after();
                        const uint64_t a = sdesc_sw128(sb + C::Q0 + (PAIR ? s * C::TILE : 0), 16, 1024);
                        const uint64_t b = sdesc_sw128(sb + C::K0 + st * C::TILE, 16, 1024);
                        if (D == 128)
                            umma_qk_k128(tm + s * 128, a, b, IQK);
                        else
                            umma_qk_k64(tm + s * 128, a, b, IQK);
                        umma_commit_elect(&sfull[s]);
                        if (!PAIR || s == 1) umma_commit_elect(&bars.kempty[st]);
                        pe[s] = e;
                        pfirst[s] = PAIR ? li == 0 : li < 2;
                        pfix[s] = fix;
                    }
                }
                for (int s = 0; s < 2 && ok; ++s)
                    if (pe[s] >= 0 && !pv(s)) ok = false;
                ro.unit_done(k);
            }
            umma_commit_elect(bars.drain);
            mbar_wait(bars.drain, 0);
        }
    } else if (warp < 12) {
        regs_dec<C::R_ROT>();
        rotate_keys<C>(ro);
    } else {
        regs_inc<C::R_SOFT>();
        // ------------------------------------------------------ softmax
        constexpr int bid = 2;  // named barrier of both warpgroups
        const int h = (warp - 12) >> 2, quad = warp & 3, lrow = quad * 32 + lane;  // half of the keys; TMEM lane
        const int pid = 3 + quad;  // named barrier of the two warps that share rows
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
        const float* ksc = reinterpret_cast<const float*>(smem + C::KSC);
        float2* xch = reinterpret_cast<float2*>(smem + C::XCH);
        float* tops = reinterpret_cast<float*>(smem + C::TOP);
        const int gshift = min(p.page_shift, 7);
        const unsigned all_pages = ro.all_pages();
        int e = 0, nu = 0;
        int done = 0, done2 = 0;  // tasks of the stream at hand, of the other
        // a wait that ran out is carried to the next barrier, where the warps that meet
        // there stop together
        bool ok = true;
        for (;; ++nu) {
            ok = ro.unit_wait(nu, 0x536);
            UnitPtr ud = ro.unit(nu);
            if (ok && ud->rows == 0) {
                named_or(bid, 256, false);  // meets a warp that gave up waiting for the unit
                break;
            }
            const unsigned char* un = smem + C::UNIT + (nu & 1) * C::UBYTES;
            const int* depth = reinterpret_cast<const int*>(un + C::U_DEPTH);
            const float* cqs = reinterpret_cast<const float*>(un + C::U_CQ) + lrow;
            const unsigned long long* ancs = reinterpret_cast<const unsigned long long*>(un + C::U_ANC) + lrow;
            ok = ok && ro.wait(&bars.uready[nu & 1], (nu >> 1) & 1, 0x531);
            // state of the row of the stream at hand and of the other's; they swap after every task
            float ref = kNoRef, l = 0.f, ref2 = kNoRef, l2 = 0.f;
            float cq = cqs[0], cq2 = cqs[PAIR ? 128 : 0];
            int tasks = 0;
            auto swap_streams = [&] {
                float f = ref; ref = ref2; ref2 = f;
                f = l; l = l2; l2 = f;
                f = cq; cq = cq2; cq2 = f;
                const int d = done; done = done2; done2 = d;
            };
            const int L = ud->L, T = ud->T, near = L + T - 1 - ud->w0;
            const int far = ud->ng > 1 ? -1 : (int)max(-1ll, (long long)L - ud->w0 - (KT - 1));
            bool alive = true;  // of the two warps that share rows
            for (UnitItems it(ud); alive && it.left > 0; it.next(), ++e) {
                const int g = it.g, j0 = it.tile * KT;
                // both streams take the tile, or they take tiles in turn
#pragma unroll 1
                for (int task = 0; task < (PAIR ? 2 : 1); ++task) {
                    const int s = tasks & 1;
                    const uint32_t s_col = lanes + s * 128 + h * 64;
                    ok = ok && ro.wait(&sfull[s], done & 1, 0x532);
                    tc_fence_after();
                    const unsigned have = ro.note()[e % INFO];
                    const volatile unsigned* flags = reinterpret_cast<const volatile unsigned*>(smem + C::SCALED) + (e % INFO) * 8;
                    unsigned any_scaled = 0;  // one flag per rotation warp of the tile
#pragma unroll
                    for (int w = 0; w < C::ROT / 32; ++w) any_scaled |= flags[w];
                    const bool drafted = j0 + KT > L || have != all_pages;
                    const bool masked = drafted || (g == 0 ? j0 <= near : j0 > far);
                    uint32_t pk[KT / 4], rest[16 * PARTS];
                    float sum;
                    // Weights at the reference as it is.  If they sum to 2^kExceed at most, no
                    // logit passed it by kExceed; else some row's reference moves and the
                    // scores are read once more.  (With the row's largest logit taken first
                    // on every tile, 64 nodes at 8 x 128K took 2.00 ms instead of 1.69.)
                    bool moved = tasks < 2;  // a stream's first tile sets its reference
#pragma unroll 1
                    for (;;) {
                        float x[KT / 2];
                        {
                            uint32_t t0[32], t1[32];
                            tmem_ld32(s_col, t0);
                            tmem_ld32(s_col + 32, t1);
                            tmem_wait_ld();
#pragma unroll
                            for (int u = 0; u < 32; ++u) {
                                x[u] = __uint_as_float(t0[u]);
                                x[32 + u] = __uint_as_float(t1[u]);
                            }
                        }
                        // key rows that were scaled by a power of two (paged_tc_roles.cuh): the
                        // whole factor here, in place of cq
                        if (any_scaled) {
                            asm volatile("" ::: "memory");
                            const float4* k4 = reinterpret_cast<const float4*>(ksc + (e % INFO) * KT + h * 64);
#pragma unroll
                            for (int u = 0; u < KT / 2; u += 4) {
                                const float4 f = k4[u / 4];
                                x[u] *= logit_factor(cq, f.x);
                                x[u + 1] *= logit_factor(cq, f.y);
                                x[u + 2] *= logit_factor(cq, f.z);
                                x[u + 3] *= logit_factor(cq, f.w);
                            }
                        }
                        const float cf = any_scaled ? 1.f : cq;
                        // what does not belong to this row and item at -inf
                        if (masked) {
                            asm volatile("" ::: "memory");  // a branch, not predication: most tiles skip this
                            const int row = (PAIR ? s * 128 : 0) + lrow, k0 = j0 + h * 64;  // first key of the half
                            const int lim = reinterpret_cast<const int*>(un + C::U_LIM)[row];
                            const int G = reinterpret_cast<const int*>(un + C::U_QG)[row];
                            // committed keys: those past the border (exact phase) or up to it
                            // (remote phase of this row's group size), before row L
                            const int cut = lim < k0 ? 0 : lim - k0 + 1;  // keys [0, cut) of the half are remote
                            const int c0 = L - k0;                        // keys [0, c0) are committed
                            auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; };
                            unsigned long long keep = below(cut);
                            keep = g == 0 ? ~keep : (G == g ? keep : 0ull);
                            keep &= below(c0);
                            if (drafted) {
                                const unsigned long long anc = ancs[PAIR ? s * 128 : 0];
                                unsigned long long nodes = 0;  // drafted nodes this row attends in this phase
#pragma unroll 1
                                for (int v = 0; v < T; ++v) {
                                    const bool local = L + depth[v] > lim;
                                    const bool in = g == 0 ? local : (!local && G == g);
                                    nodes |= (unsigned long long)(in && ((anc >> v) & 1)) << v;
                                }
                                // node v is key c0 + v
                                if (c0 > -64 && c0 < 64) keep |= c0 >= 0 ? nodes << c0 : nodes >> -c0;
                                if (have != all_pages) {
                                    unsigned long long there = 0;
#pragma unroll 1
                                    for (int u = 0; u < 64; ++u) there |= (unsigned long long)((have >> ((h * 64 + u) >> gshift)) & 1u) << u;
                                    keep &= there;
                                }
                            }
                            const uint32_t b0 = (uint32_t)keep, b1 = (uint32_t)(keep >> 32);
#pragma unroll
                            for (int u = 0; u < 32; ++u) {
                                x[u] = (b0 >> u) & 1 ? x[u] : -INFINITY;
                                x[32 + u] = (b1 >> u) & 1 ? x[32 + u] : -INFINITY;
                            }
                            __syncwarp();
                        }
                        if (moved) {
                            asm volatile("" ::: "memory");
                            float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                            for (int u = 4; u < KT / 2; u += 8) {
                                m4[0] = fmax3(m4[0], x[u], x[u + 1]);
                                m4[1] = fmax3(m4[1], x[u + 2], x[u + 3]);
                                if (u + 4 < KT / 2) {
                                    m4[2] = fmax3(m4[2], x[u + 4], x[u + 5]);
                                    m4[3] = fmax3(m4[3], x[u + 6], x[u + 7]);
                                }
                            }
                            const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                            // logits in log2 units: x cf, cf > 0 a power of two times the scale;
                            // both halves of the row's keys follow.  One place per stream: a
                            // unit's first two tasks come here without an agreement between them,
                            // so the other warp may already write the second task's maximum while
                            // this one reads the first's.  (From the third on, the agreement that
                            // ends a task's first pass lies between a read and the next write.)
                            float* const mine = tops + (s * 2 + h) * 128 + lrow;
                            *mine = top;
                            named_sync(pid, 64);
                            const float mt = fmaxf(top, mine[h ? -128 : 128]) * cf;
                            // (64 weights that sum to more than 2^kExceed hold one above 2^(kExceed - 6))
                            const bool resc = mt > ref + (kExceed - 6.5f);
                            float alpha = 1.f;
                            if (resc) {
                                alpha = ex2_approx(ref - (mt + kAbove));
                                ref = mt + kAbove;
                                l *= alpha;
                            }
                            // O (a half of its columns each) follows before any of this tile's P is published
                            if (tasks > 1 && __any_sync(0xffffffffu, resc)) {
                                ok = ro.wait(&pvdone[s], (done - 1) & 1, 0x533);
                                tc_fence_after();
                                const uint32_t o_col = lanes + 256 + s * 128 + h * (D / 2);
#pragma unroll 1
                                for (int cc = 0; cc < D / 2; cc += 16) {
                                    uint32_t tt[16];
                                    tmem_ld16(o_col + cc, tt);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int u = 0; u < 16; ++u) tt[u] = __float_as_uint(__uint_as_float(tt[u]) * alpha);
                                    tmem_st16(o_col + cc, tt);
                                }
                                tmem_wait_st();
                            }
                        }
                        const float2 sl = make_float2(cf, cf), nm = make_float2(-ref, -ref);
                        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
                        for (int u = 0; u < KT / 2; u += 4) {
                            const float2 y0 = fma2(make_float2(x[u], x[u + 1]), sl, nm);
                            const float2 y1 = fma2(make_float2(x[u + 2], x[u + 3]), sl, nm);
                            const float2 p0 = make_float2(ex2_approx(y0.x), ex2_approx(y0.y));
                            const float2 p1 = make_float2(ex2_approx(y1.x), ex2_approx(y1.y));
                            acc0 = add2(acc0, p0);
                            acc1 = add2(acc1, p1);
                            if (u < 32 * PARTS) {
                                pk[u >> 1] = split_weights(p0.x, p0.y, rest[u >> 1]);
                                pk[(u >> 1) + 1] = split_weights(p1.x, p1.y, rest[(u >> 1) + 1]);
                            } else {
                                pk[u >> 1] = pack_bf16x2(p0.x, p0.y);
                                pk[(u >> 1) + 1] = pack_bf16x2(p1.x, p1.y);
                            }
                        }
                        sum = (acc0.x + acc0.y) + (acc1.x + acc1.y);
                        if (moved || !named_or(pid, 64, !(sum <= kSumMax) || !ok)) break;
                        if (named_or(pid, 64, !ok)) {
                            alive = false;
                            break;
                        }
                        moved = true;
                    }
                    if (!alive) break;
                    // the stream's last P V finished before this tile's Q K^T (issued later by
                    // the same issuer), so each half of P may go over its half of S
                    tmem_st32(s_col, pk);
                    tmem_st16(s_col + 32, rest);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&pfull[s]);
                    l += sum;
                    ++done;
                    ++tasks;
                    swap_streams();
                }
            }
            // ---- the unit's piece is complete
            if (tasks & 1) swap_streams();  // back to stream 0 first
            if (ok && tasks > 0) ok = ro.wait(&pvdone[0], (done - 1) & 1, 0x535);
            if (ok && tasks > 1) ok = ro.wait(&pvdone[1], (done2 - 1) & 1, 0x537);
            xch[h * 128 + lrow] = make_float2(l, l2);
            tc_fence_before();
            if (named_or(bid, 256, !ok)) break;
            tc_fence_after();
            {
                const float2 o = xch[(h ^ 1) * 128 + lrow];
                l += o.x;
                l2 += o.y;
            }
            float w0 = 1.f, w1 = 0.f;  // weights of the streams' O
            if (!PAIR) {
                const float top = fmaxf(ref, ref2);
                w0 = ref == kNoRef ? 0.f : ex2_approx(ref - top);
                w1 = ref2 == kNoRef ? 0.f : ex2_approx(ref2 - top);
                l = w0 * l + w1 * l2;
                ref = top;
            }
            const int i0 = ud->i0, r0 = ud->r0, kvh = ud->kvh, rows = ud->rows;
            const bool whole = i0 == 0 && ud->i1 == ud->items;
            const unsigned long long all_bad = ud->bad;
#pragma unroll 1
            for (int s = 0; s < (PAIR ? 2 : 1); ++s) {
                const int row = s * 128 + lrow;
                const bool live = row < rows;
                const unsigned long long bad = all_bad & ancs[s * 128];
                const int node = (r0 + row) / p.group, hd = kvh * p.group + (r0 + row) % p.group;
                float* part = reinterpret_cast<float*>(p.workspace + kPagedHeader) +
                              (((size_t)blockIdx.x * 2 + (i0 == 0 ? 1 : 0)) * NROWS + row) * (D + 4);
                __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.out) + ((size_t)(ud->n0 + node) * p.Hq + hd) * D;
                const float inv = 1.f / l;
#pragma unroll 1
                for (int cb = h * (D / 2); cb < (h + 1) * (D / 2); cb += 16) {
                    uint32_t a[16], b[16];
                    tmem_ld16(lanes + 256 + s * 128 + cb, a);
                    if (!PAIR) tmem_ld16(lanes + 256 + 128 + cb, b);
                    tmem_wait_ld();
                    float v[16];
#pragma unroll
                    for (int u = 0; u < 16; ++u) {
                        v[u] = __uint_as_float(a[u]);
                        if (!PAIR)  // a stream without a key of this row holds no values
                            v[u] = (w0 != 0.f ? w0 * v[u] : 0.f) + (w1 != 0.f ? w1 * __uint_as_float(b[u]) : 0.f);
                    }
                    if (live && bad) {
                        // infinities and NaN of drafted rows this node attends
                        for (unsigned long long rest = bad; rest; rest &= rest - 1) {
                            const int r = ud->L + __ffsll((long long)rest) - 1;
                            const int page = p.table[(size_t)ud->b * p.max_pages + (r >> p.page_shift)];
                            const __nv_bfloat16* vr = static_cast<const __nv_bfloat16*>(p.vc) +
                                                      (((size_t)page * p.Hkv + kvh) * p.page_size + (r & (p.page_size - 1))) * D + cb;
#pragma unroll
                            for (int u = 0; u < 16; ++u) {
                                const float f = __bfloat162float(vr[u]);
                                if (!(fabsf(f) < INFINITY)) v[u] += f;
                            }
                        }
                    }
                    if (live && whole) {
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            *reinterpret_cast<uint4*>(orow + cb + q * 8) =
                                make_uint4(pack_bf16x2(v[8 * q] * inv, v[8 * q + 1] * inv), pack_bf16x2(v[8 * q + 2] * inv, v[8 * q + 3] * inv),
                                           pack_bf16x2(v[8 * q + 4] * inv, v[8 * q + 5] * inv), pack_bf16x2(v[8 * q + 6] * inv, v[8 * q + 7] * inv));
                    } else if (live) {
#pragma unroll
                        for (int u = 0; u < 16; u += 4)
                            *reinterpret_cast<float4*>(part + cb + u) = make_float4(v[u], v[u + 1], v[u + 2], v[u + 3]);
                    }
                }
                if (live && !whole && h == 0)
                    *reinterpret_cast<float2*>(part + D) = make_float2(ref == kNoRef ? -INFINITY : ref, l);
                ref = ref2;
                l = l2;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.ufree[nu & 1]);
            named_sync(bid, 256);  // O and xch are read before the next unit overwrites them
            ro.unit_done(nu);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, int NROWS>
cudaError_t run_one(const PagedProblem& p, const Launch& ln, cudaStream_t st, int* grid)
{
    CUtensorMap tk, tv;
    cudaError_t e;
    const int planes = p.num_pages * p.Hkv, box = std::min(p.page_size, KT);
    if ((e = tc::make_map(&tk, p.kc, D, p.page_size, p.page_size, planes, box)) != cudaSuccess) return e;
    if ((e = tc::make_map(&tv, p.vc, D, p.page_size, p.page_size, planes, box)) != cudaSuccess) return e;
    constexpr int smem = RowCfg<D, NROWS>::TOTAL;
    auto kern = decode_paged_rows_kernel<D, NROWS>;
    static PerDevice once;
    int nsm = 0;
    e = once.get(&nsm, [&](int* n, int dev) {
        cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        cudaFuncAttributes a;
        if (err == cudaSuccess) err = cudaFuncGetAttributes(&a, kern);
        // fewer registers at launch would leave setmaxnreg waiting
        using C = RowCfg<D, NROWS>;
        if (err == cudaSuccess && a.numRegs * C::THREADS < (C::R_PROD + 2 * C::R_ROT + 2 * C::R_SOFT) * 128)
            err = cudaErrorInvalidKernelImage;
        return err == cudaSuccess ? cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev) : err;
    });
    if (e != cudaSuccess) return e;
    *grid = std::min(nsm, kTcCtas);
    kern<<<*grid, RowCfg<D, NROWS>::THREADS, smem, st>>>(tk, tv, p, ln);
    return cudaGetLastError();
}

}  // namespace

cudaError_t run_rows(const PagedProblem& p, int d, int rows, const Launch& ln, cudaStream_t st, int* grid)
{
    if (d == 64) return rows <= 128 ? run_one<64, 128>(p, ln, st, grid) : run_one<64, 256>(p, ln, st, grid);
    return rows <= 128 ? run_one<128, 128>(p, ln, st, grid) : run_one<128, 256>(p, ln, st, grid);
}

}  // namespace ptc

// Query rows of a unit: the smallest capacity that holds a request's rows of one kv
// head, 256 for more (several units then).
int paged_tc_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 128 ? 128 : 256; }

size_t paged_tc_workspace(int rows, int d)
{
    return (size_t)ptc::kTcCtas * 2 * paged_tc_rows(rows) * (d + 4) * sizeof(float);
}

cudaError_t launch_decode_paged_tc(const PagedProblem& p, int d, cudaStream_t s, int* grid)
{
    const ptc::Launch ln{p.dev_error, p.wait_cycles > 0 ? p.wait_cycles : kPrefillWaitCycles, p.inject, 1};
    const int rows = paged_tc_rows(p.max_nodes * p.group);
    return rows <= 32 ? ptc::run_cols(p, d, rows, ln, s, grid) : ptc::run_rows(p, d, rows, ln, s, grid);
}

}  // namespace jl
