// decode_paged_tc.cu -- bf16 decode over a paged raw-key cache on the tensor
// cores: one new row or a tree of drafted rows per request (mathematics and
// work plan: decode_paged.cu, paged_common.cuh).
//
// A unit is (request, kv head, up to RT query rows); its keys come in tiles of
// 128.  Per tile, with the keys as the 128 rows of the first product so that its
// cost follows the number of query rows:
//   S^T [128 keys x RT]  = K_rot [128 x d] Q_rot^T [d x RT]   (fp16 operands)
//   O^T [d x RT]        += V^T [d x 128] P^T [128 x RT]       (bf16 operands)
// both accumulated in fp32 in tensor memory.  A softmax thread owns one key (one
// TMEM lane) and walks the RT columns, so the weights of a key leave as whole
// 16-byte chunks; row sums stay per thread until the unit ends.  The running
// maximum of a column only has to be near: weights are fp32 / bf16, whose range is
// far wider than the 2^40 that logits may rise by before it is taken again (kAbove),
// so each tile costs one vote of the 128 threads, and only a tile that passes the
// reference takes exact column maxima and rescales O and the sums.
//
// Warp roles:
//   warp 0      K producer: page numbers of a tile's rows, one TMA box per page
//   warp 3      V producer
//   warp 1      MMA issuer
//   warp 2      TMEM allocation
//   warps 4-11  per unit: the tree, positions, query scales; per phase: the rotated
//               queries; per tile: keys rotated in shared memory, in place (angles
//               advance from row to row); on a request's last tiles, value rows
//               that do not exist are cleared
//   warps 12-.. softmax, one warpgroup per CPT columns
// Every wait on a barrier is bounded as in the prefill kernels.
#include <algorithm>

#include "paged_common.cuh"
#include "prefill_tc_common.cuh"

namespace jl {
namespace ptc {

constexpr int KT = 128;
constexpr int kTcCtas = 148;
constexpr int INFO = 8;             // ring of per-item notes: a role is at most NSK + 2 items ahead of another
// Reference of a column (log2 units): its largest logit so far plus kAbove when it
// was last set; it is set again once a logit passes it by kExceed.  Weights then lie
// in (0, 2^kExceed], the largest of them at 2^-kAbove or above: fp32 and bf16 keep
// their relative precision over all of that, a weight 2^-100 of the largest is still
// a normal number, and only a logit that beats everything before it by 40 octaves
// costs a rescale.
constexpr float kAbove = 24.f, kExceed = 16.f;
constexpr float kNoRef = -1e30f;    // reference of a column before its first key

template <int D, int NCOL>
struct Cfg {
    static constexpr int NSK = D == 64 ? 6 : NCOL <= 64 ? 3 : 2, NSV = D == 64 ? 4 : 2;  // 16 / 32 KB stages
    static constexpr int NPV = NCOL <= 64 ? 64 : 128;  // columns of the second product (one swizzle atom is 64 wide)
    static constexpr int NWG = NCOL <= 32 ? 1 : 2, CPT = NCOL / NWG;
    static constexpr int NP = NCOL <= 64 ? 2 : 1;      // P buffers
    static constexpr int THREADS = 384 + 128 * NWG;
    // the two rotation warpgroups take tiles in turn (one's latencies under the
    // other's arithmetic) where the ring has room for two at work and one on its
    // way, else they share each tile
    static constexpr bool ALT = NSK >= 3;
    static constexpr int ROT = ALT ? 128 : 256;  // rotation threads per tile
    static constexpr int ATOMS = D / 64;
    static constexpr int TILE = KT * D * 2, ATOM_K = KT * 128, ATOM_Q = NCOL * 128;
    static constexpr int K0 = 0, V0 = K0 + NSK * TILE, P0 = V0 + NSV * TILE, PBYTES = KT * NPV * 2;
    static constexpr int Q0 = P0 + NP * PBYTES, QBYTES = NCOL * D * 2;
    static constexpr int UNIT = Q0 + (QBYTES + 1023) / 1024 * 1024;
    // unit notes, double buffered: per column ancestors, position - w0, group size, logit scale
    static constexpr int U_ANC = 0, U_DEPTH = U_ANC + NCOL * 8, U_LIM = U_DEPTH + kMaxNodes * 4, U_QG = U_LIM + NCOL * 4;
    static constexpr int U_CQ = U_QG + NCOL * 4, U_BAD = U_CQ + NCOL * 4, UBYTES = U_BAD + 16;
    static constexpr int M0 = UNIT + 2 * UBYTES;            // [NCOL] column references
    static constexpr int QS = M0 + NCOL * 4;                // [NCOL] query scales, [NCOL] positions: scratch of the unit set-up
    static constexpr int PAR = QS + NCOL * 8;               // [64] parents, [64] node ancestors
    static constexpr int RED = PAR + kMaxNodes * 12;        // [NWG][4][CPT] column maxima / sums
    static constexpr int KSC = RED + NWG * 4 * CPT * 4;     // [INFO][128] inverse key scales
    static constexpr int TURNS = KSC + INFO * KT * 4;       // [D / 2] phase constants (hi, lo)
    static constexpr int NOTE = TURNS + D / 2 * 8;          // [INFO] mask of the pages present
    static constexpr int PLAN = (NOTE + INFO * 4 + 15) / 16 * 16;
    static constexpr int SCAN = PLAN + (int)sizeof(PiecePlan);
    static constexpr int BAR = SCAN + (THREADS / 32 + 1) * 8;
    static constexpr int NBARS = 3 * NSK + 3 * NSV + 6 + 4 + 2;
    static constexpr int END = BAR + NBARS * 8 + 16;
    static constexpr int TOTAL = END + 1024;
    static_assert(TOTAL <= 232448, "shared memory");
    // Registers per thread after setmaxnreg (two softmax warpgroups only: 640
    // threads launch with 96): producers and issuer, rotation, softmax.  An
    // increase draws on what the block was launched with.
    static constexpr int R_PROD = CPT == 64 ? 40 : 56, R_ROT = CPT == 64 ? 88 : 96, R_SOFT = CPT == 64 ? 128 : 112;
    static_assert(NWG == 1 || (R_PROD + 2 * R_ROT + 2 * R_SOFT) * 128 <= THREADS * 96, "register split");
    static __device__ __forceinline__ void producer_regs() { if (NWG == 2) regs_dec<R_PROD>(); }
    static __device__ __forceinline__ void rotation_regs() { if (NWG == 2) regs_dec<R_ROT>(); }
    static __device__ __forceinline__ void softmax_regs() { if (NWG == 2) regs_inc<R_SOFT>(); }
};

struct Launch {
    int* dev_error;
    long long wait_cycles;
    int inject, min_items;
};

// Units and items of this CTA's piece, walked alike by every role.
template <int RT>
struct Walk {
    long long cur, end, base;
    int b, kvh, r0, nrows, i0, i1;
    SeqPlan s;
    __device__ __forceinline__ void init(const PiecePlan& pl)
    {
        cur = pl.start;
        end = pl.end;
        base = pl.base;
        b = pl.b;
    }
    __device__ __forceinline__ bool next(const PagedProblem& p)
    {
        if (cur >= end) return false;
        s = seq_plan<KT, RT>(p, b, false);
        long long cnt = (long long)s.items * s.row_tiles * p.Hkv;
        while (cur >= base + cnt) {
            base += cnt;
            ++b;
            s = seq_plan<KT, RT>(p, b, false);
            cnt = (long long)s.items * s.row_tiles * p.Hkv;
        }
        int unit;
        div_items(cur - base, s.items, &unit, &i0);
        i1 = (int)min((long long)s.items, i0 + (end - cur));
        kvh = unit / s.row_tiles;
        r0 = (unit % s.row_tiles) * RT;
        nrows = min(RT, s.T * p.group - r0);
        cur += i1 - i0;
        return true;
    }
};

__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ bool named_or(int id, int n, bool x)
{
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"((int)x), "r"(id), "r"(n) : "memory");
    return r != 0;
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}

// One MMA (one thread issues): D[tmem] (+)= A B, operands in shared memory.
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t mag16(uint32_t a) { return max(a & 0x7fffu, (a >> 16) & 0x7fffu); }

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
    constexpr int H = D / 2, CH = D / 16, NSK = C::NSK, NSV = C::NSV, CPT = C::CPT, NWG = C::NWG;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + C::BAR);
    uint64_t *kready = kfull + NSK, *kempty = kready + NSK, *vfull = kempty + NSK, *vempty = vfull + NSV;
    uint64_t *vfix = vempty + NSV, *sfull = vfix + NSV, *pfull = sfull + 2, *pvdone = pfull + 2;
    uint64_t *uready = pvdone + 2, *ufree = uready + 2, *qready = ufree + 2, *drain = qready + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    PiecePlan* plan = reinterpret_cast<PiecePlan*>(smem + C::PLAN);
    volatile unsigned* note = reinterpret_cast<volatile unsigned*>(smem + C::NOTE);          // [INFO]
    float* ksc = reinterpret_cast<float*>(smem + C::KSC);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < NSK; ++s) {
            mbar_init(&kfull[s], 1);
            mbar_init(&kready[s], C::ROT / 32);
            mbar_init(&kempty[s], 1);
        }
        for (int s = 0; s < NSV; ++s) {
            mbar_init(&vfull[s], 1);
            mbar_init(&vempty[s], 1);
            mbar_init(&vfix[s], C::ROT / 32);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sfull[s], 1);
            mbar_init(&pfull[s], 4 * NWG);
            mbar_init(&pvdone[s], 1);
            mbar_init(&uready[s], 8);
            mbar_init(&ufree[s], 4 * NWG);
        }
        mbar_init(qready, 8);
        mbar_init(drain, 1);
        *abort_flag = *reinterpret_cast<volatile int*>(ln.dev_error) != 0;  // an earlier wait ran out: no work
        fence_mbar_init();
    }
    for (int m = tid; m < H; m += C::THREADS)
        reinterpret_cast<uint2*>(smem + C::TURNS)[m] = make_uint2(p.turns.hi[m], p.turns.lo[m]);
    constexpr uint32_t TCOLS = NCOL <= 64 ? 256 : 512, TS = C::NPV;  // S at 0 and TS, O at 2 TS
    if (warp == 2) {
        tmem_alloc(tmem_slot, TCOLS);
        tmem_relinquish();
        tc_fence_before();
    }
    piece_plan<KT, NCOL, C::THREADS>(p, ln.min_items, plan, reinterpret_cast<long long*>(smem + C::SCAN));
    tc_fence_after();  // piece_plan ends with a barrier of the CTA
    const uint32_t tmem = *tmem_slot;
    const long long lim = ln.wait_cycles;
    Walk<NCOL> w;
    w.init(*plan);
    if (*abort_flag) w.cur = w.end;
#define PWAIT(bar, par, code) tc::warp_wait(bar, par, abort_flag, ln.dev_error, lim, code)

    if (warp < 4) C::producer_regs();
    if (warp == 0 || warp == 3) {
        // ------------------------------------------------------ producers
        const bool isK = warp == 0;
        const int NS = isK ? NSK : NSV;
        uint64_t* full = isK ? kfull : vfull;
        uint64_t* empty = isK ? kempty : vempty;
        const CUtensorMap* tm = isK ? &tmK : &tmV;
        unsigned char* ring = smem + (isK ? C::K0 : C::V0);
        const int box = min(p.page_size, KT);
        int e = 0;
        bool ok = true;
        while (ok && w.next(p)) {
            const int* table = p.table + (size_t)w.b * p.max_pages;
            Items item;
            item.start(w.s, w.i0);
            for (int i = w.i0; i < w.i1; ++i, ++e, item.next(w.s)) {
                const int tile = item.tile;
                // lane x looks after rows [x box, (x + 1) box) of the tile
                const int row = tile * KT + lane * box;
                const bool want = lane * box < KT && row < w.s.L + w.s.T;
                int page = -1;
                if (want) {
                    page = __ldg(table + (row >> p.page_shift));
                    if ((unsigned)page >= (unsigned)p.num_pages) {
                        record_input(p.input_error, kBadPage);
                        page = -1;
                    }
                }
                const int st = e % NS;
                if (e >= NS && !PWAIT(&empty[st], ((e / NS) - 1) & 1, isK ? 0x401 : 0x402)) { ok = false; break; }
                const unsigned have = __ballot_sync(0xffffffffu, page >= 0);
                if (lane == 0) {
                    if (isK) note[e % INFO] = have;
                    // (test hook: the first key tile is never loaded)
                    if (isK && e == 0 && ln.inject == kInjectDecodeCopy) {
                    } else if (have)
                        mbar_arrive_expect_tx(&full[st], (uint32_t)(__popc(have) * box * D * 2));
                    else
                        mbar_arrive(&full[st]);
                }
                __syncwarp();
                if (page >= 0 && !(isK && e == 0 && ln.inject == kInjectDecodeCopy)) {
                    unsigned char* dst = ring + st * C::TILE + lane * box * 128;
                    const int y = row & (p.page_size - 1), z = page * p.Hkv + w.kvh;
#pragma unroll
                    for (int a = 0; a < C::ATOMS; ++a) tma_load_3d(dst + a * C::ATOM_K, tm, a * 64, y, z, &full[st]);
                }
            }
        }
        // the copies in flight land before the CTA ends
        for (int x = max(0, e - NS); x < e; ++x)
            if (!(isK && x == 0 && ln.inject == kInjectDecodeCopy)) mbar_wait(&full[x % NS], (x / NS) & 1);
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        constexpr uint32_t IQK = idesc_f16(KT, NCOL, 0);
        constexpr uint32_t IPV = idesc_bf16(128, C::NPV, 1) | (1u << 15);  // A (V^T) and B (P^T) both MN-major
        const uint32_t sb = smem_u32(smem);
        int e = 0;
        unsigned nfix = 0;  // per stage: parity of the repaired value tiles so far
        bool ok = true;
        // O^T += V^T P^T of item x
        auto pv = [&](int x, bool first, bool fix) {
            if (!PWAIT(&pfull[x & 1], (x >> 1) & 1, 0x411)) return false;
            const int st = x % NSV;
            if (!PWAIT(&vfull[st], (x / NSV) & 1, 0x412)) return false;
            if (fix) {
                if (!PWAIT(&vfix[st], (nfix >> st) & 1, 0x413)) return false;
                nfix ^= 1u << st;
            }
            tc_fence_after();
            if (lane == 0) {
                // d = 64: the second 64-column atom of V^T is whatever follows the
                // tile; it fills lanes 64..127 of O^T, which nothing reads
                const uint64_t a = sdesc_sw128(sb + C::V0 + st * C::TILE, C::ATOM_K, 1024);
                const uint64_t bd = sdesc_sw128(sb + C::P0 + (x % C::NP) * C::PBYTES, C::ATOM_K, 1024);
#pragma unroll
                for (int k = 0; k < KT / 16; ++k)
                    umma_ss(tmem + 2 * TS, a + 128 * k, bd + 128 * k, IPV, !(first && k == 0));
                umma_commit(&vempty[st]);
                umma_commit(&pvdone[x & 1]);
            }
            __syncwarp();
            return true;
        };
        bool pend = false, pfirst = false, pfix = false;
        int phases = 0;
        const unsigned all_pages = (1u << (KT / min(p.page_size, KT))) - 1;
        while (ok && w.next(p)) {
            Items item;
            item.start(w.s, w.i0);
            int gcur = -1;
            for (int i = w.i0; i < w.i1; ++i, ++e, item.next(w.s)) {
                const int tile = item.tile, st = e % NSK;
                if (item.g != gcur) {
                    gcur = item.g;
                    if (!PWAIT(qready, phases & 1, 0x415)) { ok = false; break; }
                    ++phases;
                }
                if (!PWAIT(&kready[st], (e / NSK) & 1, 0x414)) { ok = false; break; }
                const bool fix = (tile + 1) * KT > w.s.L || note[e % INFO] != all_pages;
                tc_fence_after();
                if (lane == 0) {
                    const uint64_t a = sdesc_sw128(sb + C::K0 + st * C::TILE, 16, 1024);
                    const uint64_t bq = sdesc_sw128(sb + C::Q0, 16, 1024);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        umma_ss(tmem + (e & 1) * TS, a + (k >> 2) * (C::ATOM_K / 16) + (k & 3) * 2,
                                bq + (k >> 2) * (C::ATOM_Q / 16) + (k & 3) * 2, IQK, k != 0);
                    umma_commit(&kempty[st]);
                    umma_commit(&sfull[e & 1]);
                }
                __syncwarp();
                if (pend && !pv(e - 1, pfirst, pfix)) { ok = false; break; }
                pend = true;
                pfirst = i == w.i0;
                pfix = fix;
            }
        }
        if (ok && pend) pv(e - 1, pfirst, pfix);
        if (lane == 0) umma_commit(drain);
        __syncwarp();
        mbar_wait(drain, 0);
    } else if (warp >= 4 && warp < 12) {
        // ------------------------------------------------------ rotation
        C::rotation_regs();
        const int t = tid - 128, rt = t & (C::ROT - 1);  // thread of the role, of the tile
        const int group = C::ALT ? t >> 7 : 0;
        constexpr int RPT = KT * CH / C::ROT;          // rows per thread of a tile: 128 rows x CH chunk pairs
        const int c = t % CH, row0 = (rt / CH) * RPT;
        const uint4* turns = reinterpret_cast<const uint4*>(smem + C::TURNS) + c * 4;  // the thread's 8 frequencies
        float2 stc[4], sts[4];                         // cos, sin of one position step, as frequency pairs
        auto angles = [&](uint32_t f, float2 (&cs)[4], float2 (&sn)[4]) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint4 w2 = turns[u];
                rope_cs_fast(f, w2.x, w2.y, cs[u].x, sn[u].x);
                rope_cs_fast(f, w2.z, w2.w, cs[u].y, sn[u].y);
            }
        };
        angles(1u, stc, sts);
        // 8 pairs (lo.x holds dimensions 0, 1 of the chunk, hi.x their partners, ...)
        // turned by (cs, sn), as fp16
        auto turn = [&](uint4& lo, uint4& hi, const float2 (&cs)[4], const float2 (&sn)[4]) {
            uint32_t* a = &lo.x;
            uint32_t* b = &hi.x;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float2 x = make_float2(bf16_lo(a[u]), bf16_hi(a[u])), y = make_float2(bf16_lo(b[u]), bf16_hi(b[u]));
                const float2 ny = make_float2(__uint_as_float((b[u] << 16) + 0x80000000u),
                                              __uint_as_float((b[u] & 0xffff0000u) ^ 0x80000000u));
                const float2 r0 = fma2(ny, sn[u], mul2(x, cs[u])), r1 = fma2(y, cs[u], mul2(x, sn[u]));
                a[u] = pack_f16x2(r0.x, r0.y);
                b[u] = pack_f16x2(r1.x, r1.y);
            }
        };
        auto absmax8 = [](const uint4& a, const uint4& b) {
            return absmax2(absmax2(absmax2(a.x, a.y), absmax2(a.z, a.w)), absmax2(absmax2(b.x, b.y), absmax2(b.z, b.w)));
        };
        auto scale8 = [](uint4& a, float sc) {  // exact: a power of two (elements far below the row's largest may vanish)
            a.x = pack_bf16x2(bf16_lo(a.x) * sc, bf16_hi(a.x) * sc);
            a.y = pack_bf16x2(bf16_lo(a.y) * sc, bf16_hi(a.y) * sc);
            a.z = pack_bf16x2(bf16_lo(a.z) * sc, bf16_hi(a.z) * sc);
            a.w = pack_bf16x2(bf16_lo(a.w) * sc, bf16_hi(a.w) * sc);
        };
        const int gshift = min(p.page_shift, 7);
        const unsigned all_pages = (1u << (KT >> gshift)) - 1;
        int* par = reinterpret_cast<int*>(smem + C::PAR);
        unsigned long long* nanc = reinterpret_cast<unsigned long long*>(par + kMaxNodes);
        float* qsc = reinterpret_cast<float*>(smem + C::QS);
        int* qpos = reinterpret_cast<int*>(qsc + NCOL);
        int e = 0, nu = 0;
        // A wait that runs out in one warp must not leave the others at a barrier:
        // the warps meet once per unit (and once after the last) and stop together
        // if any of them gave up.
        bool ok = true, agreed = false;
        while (ok && w.next(p)) {
            unsigned char* un = smem + C::UNIT + (nu & 1) * C::UBYTES;
            int* depth = reinterpret_cast<int*>(un + C::U_DEPTH);
            int* lim0 = reinterpret_cast<int*>(un + C::U_LIM);
            int* qG = reinterpret_cast<int*>(un + C::U_QG);
            float* cq = reinterpret_cast<float*>(un + C::U_CQ);
            unsigned long long* canc = reinterpret_cast<unsigned long long*>(un + C::U_ANC);
            unsigned long long* bad = reinterpret_cast<unsigned long long*>(un + C::U_BAD);
            int* big = reinterpret_cast<int*>(bad + 1);
            // the softmax is done with unit nu - 2, the tensor cores with the
            // queries of unit nu - 1
            ok = (nu < 2 || PWAIT(&ufree[nu & 1], ((nu >> 1) - 1) & 1, 0x421)) &&
                 (e == 0 || PWAIT(&kempty[(e - 1) % NSK], ((e - 1) / NSK) & 1, 0x422));
            if ((agreed = named_or(1, 256, !ok))) break;
            if (t < w.s.T) {
                int x = t - 1;
                if (p.parents) {
                    x = p.parents[w.s.n0 + t];
                    if (x < -1 || x >= t) {
                        record_input(p.input_error, kBadParent);
                        x = -1;
                    }
                }
                par[t] = x;
            }
            if (t == 0) {
                *bad = 0;
                *big = 0;
            }
            named_sync(1, 256);
            if (t < w.s.T) {
                unsigned long long m = (2ull << t) - 1;
                if (p.parents) {
                    m = 0;
                    for (int x = t; x >= 0; x = par[x]) m |= 1ull << x;
                }
                nanc[t] = m;
                depth[t] = __popcll(m) - 1;
            }
            named_sync(1, 256);
            if (t < NCOL) {
                int x = 0, G = 0;
                float inv = 0.f, sc = 0.f;
                unsigned long long up = 0;
                if (t < w.nrows) {
                    const int node = (w.r0 + t) / p.group, hd = w.kvh * p.group + (w.r0 + t) % p.group;
                    x = w.s.L + depth[node];
                    G = x / p.w_pre + 1;
                    up = nanc[node];
                    // the query times a power of two that brings its largest element
                    // into [2^13, 2^14); the logits times the inverse
                    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                                    ((size_t)(w.s.n0 + node) * p.Hq + hd) * D);
                    uint32_t mx = 0;
                    float l1 = 0.f;
#pragma unroll 4
                    for (int k = 0; k < D / 8; ++k) {
                        const uint4 v = q[k];
                        mx = absmax2(mx, absmax2(absmax2(v.x, v.y), absmax2(v.z, v.w)));
                        l1 += fabsf(bf16_lo(v.x)) + fabsf(bf16_hi(v.x)) + fabsf(bf16_lo(v.y)) + fabsf(bf16_hi(v.y)) +
                              fabsf(bf16_lo(v.z)) + fabsf(bf16_hi(v.z)) + fabsf(bf16_lo(v.w)) + fabsf(bf16_hi(v.w));
                    }
                    const int ex = tc::range_exp(mag16(mx));
                    sc = tc::pow2i(ex);
                    inv = tc::pow2i(-ex) * p.scale_log2;
                    // keys rounded to fp16 as they are err by up to 2^-25 where fp16 is
                    // subnormal; with an L1 norm this large that could reach 2^-11 of a logit
                    if (!(l1 * p.scale_log2 * 1.4142136f <= 16384.f)) *big = 1;
                }
                qpos[t] = x;
                lim0[t] = x - w.s.w0;
                qG[t] = G;
                canc[t] = up;
                cq[t] = inv;
                qsc[t] = sc;
            }
            named_sync(1, 256);
            if (lane == 0) mbar_arrive(&uready[nu & 1]);
            const bool always = *big != 0;
            const int n = w.s.L + w.s.T;
            int gcur = -1;
            uint32_t dm = 0, ds1 = 0, ds2 = 0;  // division by the group size by multiply-shift
            Items item;
            item.start(w.s, w.i0);
            for (int i = w.i0; i < w.i1; ++i, ++e, item.next(w.s)) {
                const int g = item.g;
                if (g != gcur) {
                    // queries of this phase; the tensor cores are done with those of the last
                    if (gcur >= 0 && !PWAIT(&kempty[(e - 1) % NSK], ((e - 1) / NSK) & 1, 0x423)) { ok = false; break; }
                    gcur = g;
                    const uint32_t dv = max(g, 1);
                    const uint32_t lg = 32 - __clz(dv - 1);  // ceil(log2 dv); 0 for 1
                    dm = (uint32_t)(((((uint64_t)1 << 32) * (((uint64_t)1 << lg) - dv)) / dv) + 1);
                    ds1 = min(lg, 1u);
                    ds2 = lg > 1 ? lg - 1 : 0;
#pragma unroll 1
                    for (int x = t; x < NCOL * CH; x += 256) {
                        const int r = x / CH;  // CH divides 256: chunk x % CH = c
                        uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
                        if (r < w.nrows) {
                            const int node = (w.r0 + r) / p.group, hd = w.kvh * p.group + (w.r0 + r) % p.group;
                            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) +
                                                     ((size_t)(w.s.n0 + node) * p.Hq + hd) * D;
                            lo = *reinterpret_cast<const uint4*>(q + c * 8);
                            hi = *reinterpret_cast<const uint4*>(q + H + c * 8);
                            float2 cs[4], sn[4];
                            angles((uint32_t)qpos[r] / dv, cs, sn);
                            const float2 sc = make_float2(qsc[r], qsc[r]);
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                cs[u] = mul2(cs[u], sc);
                                sn[u] = mul2(sn[u], sc);
                            }
                            turn(lo, hi, cs, sn);
                        }
                        *reinterpret_cast<uint4*>(smem + C::Q0 + tc::sw128_off<NCOL>(r, c)) = lo;
                        *reinterpret_cast<uint4*>(smem + C::Q0 + tc::sw128_off<NCOL>(r, c + CH)) = hi;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(qready);
                }
                if (C::ALT && (e & 1) != group) continue;
                const int st = e % NSK, j0 = item.tile * KT;
                unsigned char* kt = smem + C::K0 + st * C::TILE;
                const bool drafted = j0 + KT > w.s.L;
                // turned position of a row: its place, or a drafted row's depth, over the
                // group size (rows past the end: 0, they are masked)
                auto turned = [&](int r) {
                    const int j = j0 + r;
                    uint32_t pos = (uint32_t)j;
                    if (drafted && j >= w.s.L) pos = j < n ? (uint32_t)(w.s.L + depth[j - w.s.L]) : 0u;
                    const uint32_t t1 = __umulhi(dm, pos);
                    return (t1 + ((pos - t1) >> ds1)) >> ds2;
                };
                uint32_t f = turned(row0);
                float2 cs[4], sn[4];
                angles(f, cs, sn);
                if (!PWAIT(&kfull[st], (e / NSK) & 1, 0x424)) { ok = false; break; }
                // from row to row the turned position stays or steps by one (drafted
                // rows may jump): the angles follow by the angle addition
                auto advance = [&](int r) {
                    const uint32_t fn = turned(r);
                    if (fn == f + 1) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float2 ns = make_float2(-sn[u].x, -sn[u].y);
                            const float2 nc = fma2(ns, sts[u], mul2(cs[u], stc[u]));
                            sn[u] = fma2(cs[u], sts[u], mul2(sn[u], stc[u]));
                            cs[u] = nc;
                        }
                    } else if (fn != f) {
                        angles(fn, cs, sn);
                    }
                    f = fn;
                };
#pragma unroll 1
                for (int x = 0; x < RPT; x += 2) {
                    const int r = row0 + x;
                    uint4* pa = reinterpret_cast<uint4*>(kt + tc::sw128_off<KT>(r, c));
                    uint4* pb = reinterpret_cast<uint4*>(kt + tc::sw128_off<KT>(r, c + CH));
                    uint4* pc = reinterpret_cast<uint4*>(kt + tc::sw128_off<KT>(r + 1, c));
                    uint4* pd = reinterpret_cast<uint4*>(kt + tc::sw128_off<KT>(r + 1, c + CH));
                    uint4 a0 = *pa, b0 = *pb, a1 = *pc, b1 = *pd;
                    // Keys are rounded to fp16 as they are, unless one of the warp's is too
                    // large for it (0x4700: 2^15), or the query makes small ones count: then
                    // every row is first scaled by its own power of two.
                    uint32_t m0 = absmax8(a0, b0), m1 = absmax8(a1, b1);
                    float k0 = 1.f, k1 = 1.f;
                    if (__any_sync(0xffffffffu, always || mag16(absmax2(m0, m1)) >= 0x4700u)) {
                        m0 = mag16(m0);
                        m1 = mag16(m1);
#pragma unroll
                        for (int o = 1; o < CH; o <<= 1) {
                            m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, o));
                            m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, o));
                        }
                        const int e0 = tc::range_exp(m0), e1 = tc::range_exp(m1);
                        scale8(a0, tc::pow2i(e0));
                        scale8(b0, tc::pow2i(e0));
                        scale8(a1, tc::pow2i(e1));
                        scale8(b1, tc::pow2i(e1));
                        k0 = tc::pow2i(-e0);
                        k1 = tc::pow2i(-e1);
                    }
                    if (c == 0) *reinterpret_cast<float2*>(ksc + (e % INFO) * KT + r) = make_float2(k0, k1);
                    if (x > 0) advance(r);
                    turn(a0, b0, cs, sn);
                    *pa = a0;
                    *pb = b0;
                    advance(r + 1);
                    turn(a1, b1, cs, sn);
                    *pc = a1;
                    *pd = b1;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&kready[st]);
                // value rows that do not exist count as zero: the page may hold
                // anything there, and a weight of 0 does not silence NaN.  A drafted
                // row's own infinities and NaN are cleared as well (nodes beside it
                // must not see them) and noted for the nodes that do attend it.
                const unsigned have = note[e % INFO];
                if (drafted || have != all_pages) {
                    const int sv = e % NSV;
                    if (!PWAIT(&vfull[sv], (e / NSV) & 1, 0x425)) { ok = false; break; }
                    unsigned char* vt = smem + C::V0 + sv * C::TILE;
                    constexpr int TPR = C::ROT / KT;  // threads per row
                    const int r = rt / TPR, j = j0 + r;
                    const bool there = j < n && ((have >> (r >> gshift)) & 1);
                    if (!there || j >= w.s.L) {
#pragma unroll 1
                        for (int k = rt % TPR; k < D / 8; k += TPR) {
                            uint4* v = reinterpret_cast<uint4*>(vt + tc::sw128_off<KT>(r, k));
                            if (!there) {
                                *v = make_uint4(0u, 0u, 0u, 0u);
                                continue;
                            }
                            uint4 x = *v;
                            uint32_t* y = &x.x;
                            bool hit = false;
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                if ((y[u] & 0x7f80u) == 0x7f80u) { y[u] &= 0xffff0000u; hit = true; }
                                if ((y[u] & 0x7f800000u) == 0x7f800000u) { y[u] &= 0xffffu; hit = true; }
                            }
                            if (hit) {
                                *v = x;
                                atomicOr(bad, 1ull << (j - w.s.L));
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&vfix[sv]);
                }
            }
            ++nu;
        }
        if (!agreed) named_or(1, 256, !ok);
    } else if (warp >= 12) {
        // ------------------------------------------------------ softmax
        C::softmax_regs();
        const int wg = (warp - 12) >> 2, wl = warp & 3, c0 = wg * CPT;
        const int key = wl * 32 + lane, bid = 2 + wg;
        const uint32_t tl = tmem + ((uint32_t)(32 * wl) << 16);
        float* mref = reinterpret_cast<float*>(smem + C::M0) + c0;
        float* red = reinterpret_cast<float*>(smem + C::RED) + wg * 4 * CPT;
        float l[CPT];
        int e = 0, nu = 0;
        // as above, a wait that ran out is carried to the warpgroup's next barrier,
        // where its four warps stop together
        bool ok = true, stop = false;
        const int gshift = min(p.page_shift, 7);
        const unsigned all_pages = (1u << (KT >> gshift)) - 1;
        if (tid == 384) clear_cut(p);
        while (!stop && w.next(p)) {
            const unsigned char* un = smem + C::UNIT + (nu & 1) * C::UBYTES;
            const int* depth = reinterpret_cast<const int*>(un + C::U_DEPTH);
            const int* clim = reinterpret_cast<const int*>(un + C::U_LIM) + c0;
            const int* qG = reinterpret_cast<const int*>(un + C::U_QG) + c0;
            const float* cq = reinterpret_cast<const float*>(un + C::U_CQ) + c0;
            const unsigned long long* canc = reinterpret_cast<const unsigned long long*>(un + C::U_ANC) + c0;
            ok = PWAIT(&uready[nu & 1], (nu >> 1) & 1, 0x431);
#pragma unroll
            for (int c = 0; c < CPT; ++c) l[c] = 0.f;
            if (key < CPT) mref[key] = kNoRef;
            if (named_or(bid, 128, !ok)) break;
            const int cols = min(CPT, w.nrows - c0);  // may be <= 0: nothing but the hand-over
            const int L = w.s.L, n = L + w.s.T;
            Items item;
            item.start(w.s, w.i0);
            for (int i = w.i0; i < w.i1; ++i, ++e, item.next(w.s)) {
                const int g = item.g, j0 = item.tile * KT;
                ok = ok && PWAIT(&sfull[e & 1], (e >> 1) & 1, 0x432);
                tc_fence_after();
                const unsigned have = note[e % INFO];
                // which pairs of the tile this item leaves out: some of a drafted or
                // incomplete tile's; the other branch's on the border of the window
                // (or of columns with another group size)
                const bool drafted = j0 + KT > L || have != all_pages;
                const bool masked = drafted || (g == 0 ? n - 1 - j0 >= w.s.w0 : (w.s.ng > 1 || L - (j0 + KT - 1) < w.s.w0));
                const float ks = *reinterpret_cast<volatile float*>(ksc + (e % INFO) * KT + key);
                const bool any_scaled = __any_sync(0xffffffffu, ks != 1.f);
                const int j = j0 + key, u = j - L;
                const bool there = j < n && ((have >> (key >> gshift)) & 1);
                // one bit per column: the pair belongs to this item
                uint32_t keep[(CPT + 31) / 32];
                if (masked) {
                    asm volatile("" ::: "memory");  // a branch, not predication: most tiles skip this
                    const int kpos = there ? (u < 0 ? j : L + depth[u]) : 0;
                    const unsigned long long self = u < 0 ? ~0ull : 1ull << (u & 63);
#pragma unroll
                    for (int cb = 0; cb < CPT; cb += 32) {
                        uint32_t bits = 0;
#pragma unroll 4
                        for (int c = 0; c < min(32, CPT); ++c) {
                            const bool local = kpos > clim[cb + c];
                            const bool mine = g == 0 ? local : (!local && qG[cb + c] == g);
                            bits |= (uint32_t)(mine && there && (u < 0 || (canc[cb + c] & self))) << c;
                        }
                        keep[cb / 32] = bits;
                    }
                }
                // logits of 16 columns from cb on in log2 units, minus their references;
                // what this item leaves out is -inf
                auto logits = [&](int cb, float (&y)[16], bool relative) {
                    uint32_t raw[16];
                    tmem_ld16(tl + (e & 1) * TS + c0 + cb, raw);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; ++c) y[c] = __uint_as_float(raw[c]);
                    if (any_scaled) {
                        asm volatile("" ::: "memory");
#pragma unroll
                        for (int c = 0; c < 16; ++c) y[c] *= ks;
                    }
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {
                        const float4 k4 = *reinterpret_cast<const float4*>(cq + cb + c);
                        float4 m4 = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (relative) m4 = *reinterpret_cast<const float4*>(mref + cb + c);
                        y[c] = fmaf(y[c], k4.x, -m4.x);
                        y[c + 1] = fmaf(y[c + 1], k4.y, -m4.y);
                        y[c + 2] = fmaf(y[c + 2], k4.z, -m4.z);
                        y[c + 3] = fmaf(y[c + 3], k4.w, -m4.w);
                    }
                    if (masked) {
                        asm volatile("" ::: "memory");
                        const uint32_t bits = keep[cb / 32] >> (cb & 31);
#pragma unroll
                        for (int c = 0; c < 16; ++c) y[c] = (bits >> c) & 1 ? y[c] : -INFINITY;
                    }
                };
                float y[16];
                for (;;) {
                    float top = -INFINITY;
#pragma unroll
                    for (int cb = 0; cb < CPT; cb += 16) {
                        if (cb < cols) {
                            logits(cb, y, true);
#pragma unroll
                            for (int c = 0; c < 16; c += 2) top = fmax3(top, y[c], y[c + 1]);
                        }
                    }
                    if (!named_or(bid, 128, top > kExceed || !ok)) break;
                    if (named_or(bid, 128, !ok)) {
                        stop = true;
                        break;
                    }
                    // exact column maxima of this tile; sums and O follow the new references
#pragma unroll
                    for (int cb = 0; cb < CPT; cb += 16) {
                        if (cb >= cols) break;
                        float v[16];
                        logits(cb, v, false);
                        const float m = lane_columns<true>(v, lane);
                        if (lane < 16) red[wl * CPT + cb + lane] = m;
                    }
                    named_sync(bid, 128);
                    float alpha = 1.f;
                    if (key < CPT && key < (cols + 15) / 16 * 16) {
                        const float m = fmaxf(fmaxf(red[key], red[CPT + key]), fmaxf(red[2 * CPT + key], red[3 * CPT + key]));
                        const float old = mref[key];
                        if (m > -INFINITY && m + kAbove > old) {
                            mref[key] = m + kAbove;
                            alpha = exp2f(old - (m + kAbove));
                        }
                    }
                    named_sync(bid, 128);
                    if (key < CPT) red[key] = alpha;
                    named_sync(bid, 128);
#pragma unroll
                    for (int c = 0; c < CPT; ++c) l[c] *= red[c];
                    if (i > w.i0) {
                        ok = PWAIT(&pvdone[(e - 1) & 1], ((e - 1) >> 1) & 1, 0x433);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < CPT; c += 16) {
                            if (c >= cols) break;
                            uint32_t o[16];
                            tmem_ld16(tl + 2 * TS + c0 + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * red[c + x]);
                            tmem_st16(tl + 2 * TS + c0 + c, o);
                        }
                        tmem_wait_st();
                    }
                    if (named_or(bid, 128, !ok)) {  // and red is read before it is written again
                        stop = true;
                        break;
                    }
                }
                if (stop) break;
                // weights to the P buffer, free once P V of item e - NP is done
                if (e >= C::NP) {
                    const int x = e - C::NP;
                    ok = PWAIT(&pvdone[x & 1], (x >> 1) & 1, 0x434);
                }
                unsigned char* pb = smem + C::P0 + (e % C::NP) * C::PBYTES + (c0 >> 6) * C::ATOM_K + key * 128;
#pragma unroll
                for (int cb = 0; cb < CPT; cb += 16) {
                    if (cb < cols) {
                        if (CPT > 16) logits(cb, y, true);  // else still there
#pragma unroll
                        for (int c = 0; c < 16; c += 8) {
                            uint32_t o[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const float a = ex2_approx(y[c + 2 * x]), bb = ex2_approx(y[c + 2 * x + 1]);
                                l[cb + c + 2 * x] += a;
                                l[cb + c + 2 * x + 1] += bb;
                                o[x] = pack_bf16x2(a, bb);
                            }
                            *reinterpret_cast<uint4*>(pb + (((((c0 + cb + c) & 63) >> 3) ^ (key & 7)) << 4)) =
                                make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    }
                }
                tc_fence_before();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[e & 1]);
            }
            if (stop) break;
            // ---- the unit's piece is complete
            ok = ok && PWAIT(&pvdone[(e - 1) & 1], ((e - 1) >> 1) & 1, 0x435);
            tc_fence_after();
#pragma unroll
            for (int cb = 0; cb < CPT; cb += 16) {
                float v[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) v[c] = l[cb + c];
                const float sum = lane_columns<false>(v, lane);
                if (lane < 16) red[wl * CPT + cb + lane] = sum;
            }
            if (named_or(bid, 128, !ok)) break;
            const bool whole = w.i0 == 0 && w.i1 == w.s.items;
            if (tid == 384 && w.i0 == 0 && !whole) note_cut(p, w.s, plan->per, w.cur - w.i1, w.kvh, w.r0, w.nrows);
            const unsigned long long bad = *reinterpret_cast<const volatile unsigned long long*>(un + C::U_BAD);
            float* part = reinterpret_cast<float*>(p.workspace + kPagedHeader) +
                          ((size_t)blockIdx.x * 2 + (w.i0 == 0 ? 1 : 0)) * NCOL * (D + 2);
#pragma unroll 1
            for (int cb = 0; cb < CPT; cb += 16) {
                if (cb >= cols) break;
                uint32_t o[16];
                tmem_ld16(tl + 2 * TS + c0 + cb, o);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const int c = cb + x;
                    if (c >= cols) break;
                    float val = __uint_as_float(o[x]);
                    const float sum = red[c] + red[CPT + c] + red[2 * CPT + c] + red[3 * CPT + c];
                    if (bad && key < D) {
                        // infinities and NaN of drafted rows this node attends
                        for (unsigned long long rest = bad & canc[c]; rest; rest &= rest - 1) {
                            const int row = L + __ffsll((long long)rest) - 1;
                            const int page = p.table[(size_t)w.b * p.max_pages + (row >> p.page_shift)];
                            const float v = __bfloat162float(static_cast<const __nv_bfloat16*>(p.vc)[
                                (((size_t)page * p.Hkv + w.kvh) * p.page_size + (row & (p.page_size - 1))) * D + key]);
                            if (!(fabsf(v) < INFINITY)) val += v;
                        }
                    }
                    const int r = c0 + c;
                    if (whole) {
                        const int node = (w.r0 + r) / p.group, hd = w.kvh * p.group + (w.r0 + r) % p.group;
                        if (key < D)
                            static_cast<__nv_bfloat16*>(p.out)[((size_t)(w.s.n0 + node) * p.Hq + hd) * D + key] =
                                __float2bfloat16_rn(val / sum);
                    } else {
                        if (key < D) part[(size_t)r * (D + 2) + key] = val;
                        if (key < 2) part[(size_t)r * (D + 2) + D + key] = key == 0 ? (mref[c] == kNoRef ? -INFINITY : mref[c]) : sum;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ufree[nu & 1]);
            named_sync(bid, 128);  // red and mref are read before the next unit writes them
            ++nu;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, TCOLS);
    }
#undef PWAIT
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
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    int dev = 0, nsm = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    *grid = std::min(nsm, kTcCtas);
    kern<<<*grid, Cfg<D, NCOL>::THREADS, smem, st>>>(tk, tv, p, ln);
    return cudaGetLastError();
}

}  // namespace ptc

// Columns of a unit: the smallest capacity that holds a request's query rows of
// one kv head, 128 for more (several units then).
int paged_tc_columns(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

size_t paged_tc_workspace(int rows, int d)
{
    return (size_t)ptc::kTcCtas * 2 * paged_tc_columns(rows) * (d + 2) * sizeof(float);
}

cudaError_t launch_decode_paged_tc(const PagedProblem& p, int d, cudaStream_t s, int* grid)
{
    ptc::Launch ln{p.dev_error, p.wait_cycles > 0 ? p.wait_cycles : kPrefillWaitCycles, p.inject, 1};
    const int cols = paged_tc_columns(p.max_nodes * p.group);
    if (d == 64) {
        switch (cols) {
            case 16: return ptc::run<64, 16>(p, ln, s, grid);
            case 32: return ptc::run<64, 32>(p, ln, s, grid);
            case 64: return ptc::run<64, 64>(p, ln, s, grid);
            default: return ptc::run<64, 128>(p, ln, s, grid);
        }
    }
    switch (cols) {
        case 16: return ptc::run<128, 16>(p, ln, s, grid);
        case 32: return ptc::run<128, 32>(p, ln, s, grid);
        case 64: return ptc::run<128, 64>(p, ln, s, grid);
        default: return ptc::run<128, 128>(p, ln, s, grid);
    }
}

}  // namespace jl
