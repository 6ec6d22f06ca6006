// paged_tc_roles.cuh -- the warp roles that both tensor-core kernels of the paged
// decode share: the producers of key and value tiles, the planner of units, and
// the rotation of keys and queries.  A kernel's configuration C lays out shared
// memory and says how many threads share a tile.
//
// Every wait on a barrier is bounded (an mbarrier wait gives up after a limit,
// records a code in the device error word and sets the CTA's abort flag, which
// ends every other wait); warps that meet at a named barrier agree there whether
// any of them gave up, so none is left waiting at it.
#pragma once

#include "paged_common.cuh"
#include "prefill_tc_common.cuh"

namespace jl {
namespace ptc {

constexpr int KT = 128;
constexpr int kTcCtas = 148;
// Reference of a query row (log2 units): its largest logit so far plus kAbove when it
// was last set; it is set again once a logit passes it by kExceed.  Weights then lie
// in (0, 2^kExceed], the largest of them at 2^-kAbove or above: fp32 and bf16 keep
// their relative precision over all of that, a weight 2^-100 of the largest is still
// a normal number, and only a logit that beats everything before it by 40 octaves
// costs a rescale.
constexpr float kAbove = 24.f, kExceed = 16.f;
constexpr float kNoRef = -1e30f;    // reference of a row before its first key
constexpr int UNITS = 4;            // ring of units planned ahead
constexpr int INFO = 8;             // ring of per-item notes: a role is at most NSK + 2 items ahead of another
// A unit of this CTA's piece, as the planner leaves it in shared memory for the
// other roles (read there field by field: registers are scarce).
struct UnitDesc {
    int rows;            // query rows; 0: no more units
    int L, T, n0, b;     // committed rows, nodes, first token row, request
    int kvh, r0;         // kv head, first query row
    int i0, i1;          // its items in this piece
    int gmin, ng, nR, kE0, w0, items, pad0;
    unsigned long long bad;  // drafted nodes whose value rows hold infinities or NaN (value producer)
};
typedef const volatile UnitDesc* UnitPtr;

struct Launch {
    int* dev_error;
    long long wait_cycles;
    int inject, min_items;
};

// Up to 32 query rows per unit: decode_paged_tc.cu; more: decode_paged_rows.cu.
cudaError_t run_cols(const PagedProblem& p, int d, int cols, const Launch& ln, cudaStream_t st, int* grid);
cudaError_t run_rows(const PagedProblem& p, int d, int rows, const Launch& ln, cudaStream_t st, int* grid);

// Shared memory after the tiles, from offset BASE: notes of two units (per query
// row: ancestors, position - w0, group size, logit scale; per node: depth), scratch
// of the unit set-up, rings of per-item notes, the plan and the barriers.
template <int D, int ROWS, int NSK, int NSV, int BASE, int EXTRA_BARS, int WARPS>
struct Notes {
    static constexpr int UNIT = BASE;
    static constexpr int U_ANC = 0, U_DEPTH = U_ANC + ROWS * 8, U_LIM = U_DEPTH + kMaxNodes * 4, U_QG = U_LIM + ROWS * 4;
    static constexpr int U_CQ = U_QG + ROWS * 4, U_BIG = U_CQ + ROWS * 4, UBYTES = U_BIG + 16;
    static constexpr int PAR = UNIT + 2 * UBYTES;           // [64] parents, [64] node ancestors
    static constexpr int KSC = PAR + kMaxNodes * 12;        // [INFO][128] inverse key scales
    static constexpr int TURNS = KSC + INFO * KT * 4;       // [D / 2] phase constants (hi, lo)
    static constexpr int NOTE = TURNS + D / 2 * 8;          // [INFO] mask of the pages present
    static constexpr int SCALED = NOTE + INFO * 4;          // [INFO][8] a rotation warp scaled rows of the tile
    static constexpr int PLAN = SCALED + INFO * 32;
    static constexpr int DESC = PLAN + (int)sizeof(PiecePlan);
    static constexpr int SCAN = DESC + UNITS * (int)sizeof(UnitDesc);
    static constexpr int BAR = SCAN + (WARPS + 1) * 8;
    // Landed key tiles are announced on a ring of an even number of barriers, apart
    // from the ring of stages: the two rotation warpgroups wait for every second tile,
    // and a barrier that one of them sees only every second time around would let a
    // parity wait pass a phase early.
    static constexpr int NKF = NSK + (NSK & 1);
    static constexpr int NBARS = NKF + 2 * NSK + 3 * NSV + 5 + 1 + 2 * UNITS + EXTRA_BARS;
    static constexpr int SLOT = BAR + NBARS * 8;            // TMEM address, abort flag
    static constexpr int NOTES_END = (SLOT + 16 + 15) / 16 * 16;
    static_assert(INFO > NSK + 1, "ring of per-item notes");
};

// The CTA's dynamic shared memory from its first 1024-byte boundary on.  Derived from
// the array by an offset, not by a cast through an integer, so that the compiler
// keeps seeing shared memory.
__device__ __forceinline__ unsigned char* smem_base()
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    return smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
}

// The barriers, in the order of their use.
template <class C>
struct Bars {
    uint64_t *kfull, *kready, *kempty;  // key tile landed; rotated; read by the tensor cores
    uint64_t *vfull, *vfix, *vempty;    // value tile landed; cleared where rows are missing; read
    uint64_t *uready, *ufree;           // notes of unit k (two buffers) written; done with
    uint64_t *qready;                   // queries of a phase rotated
    uint64_t *dfull, *dfree;            // unit planned; done with
    uint64_t *drain, *extra;
    __device__ __forceinline__ Bars()
    {
        kfull = reinterpret_cast<uint64_t*>(smem_base() + C::BAR);
        kready = kfull + C::NKF;
        kempty = kready + C::NSK;
        vfull = kempty + C::NSK;
        vfix = vfull + C::NSV;
        vempty = vfix + C::NSV;
        uready = vempty + C::NSV;
        ufree = uready + 2;
        qready = ufree + 2;
        dfull = qready + 1;
        dfree = dfull + UNITS;
        drain = dfree + UNITS;
        extra = drain + 1;
    }
    // one thread; C::ROT threads rotate a tile, C::ROTALL in all, C::SOFT softmax warps
    __device__ __forceinline__ void init()
    {
        for (int s = 0; s < C::NKF; ++s) mbar_init(&kfull[s], 1);
        for (int s = 0; s < C::NSK; ++s) {
            mbar_init(&kready[s], C::ROT / 32);
            mbar_init(&kempty[s], 1);
        }
        for (int s = 0; s < C::NSV; ++s) {
            mbar_init(&vfull[s], 1);
            mbar_init(&vfix[s], 1);
            mbar_init(&vempty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&uready[s], C::ROTALL / 32);
            mbar_init(&ufree[s], C::SOFT);
        }
        mbar_init(qready, C::ROTALL / 32);
        for (int s = 0; s < UNITS; ++s) {
            mbar_init(&dfull[s], 1);
            mbar_init(&dfree[s], 3 + C::ROTALL / 32 + C::SOFT);  // two producers, the issuer, rotation, softmax
        }
        mbar_init(drain, 1);
    }
};

// The items of a unit in order: the group size its keys are aliased by (0: exact
// positions) and the key tile.
struct UnitItems {
    int g, tile, left, nR, kE0, gend;
    __device__ __forceinline__ explicit UnitItems(UnitPtr u)
    {
        const int i = u->i0, rem = u->ng * u->nR;
        nR = u->nR;
        kE0 = u->kE0;
        gend = u->gmin + u->ng;
        left = u->i1 - i;
        g = 0;
        tile = kE0 + (i - rem);
        if (i < rem) {
            g = u->gmin + i / nR;
            tile = i % nR;
        }
    }
    __device__ __forceinline__ void next()
    {
        --left;
        ++tile;
        if (g != 0 && tile == nR) {
            ++g;
            tile = 0;
            if (g == gend) {
                g = 0;
                tile = kE0;
            }
        }
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

// Groups of MMAs from one elected lane of a converged warp, D[tmem] (+)= A B with both
// operands in shared memory; the descriptors of later steps are the first one's plus
// immediates (16-byte units; no carry out of the address field).  Issued one by one
// from a single thread, the 16 MMAs of a tile took 2500 cycles, most of a tile's time.
#define JL_SS(AO, BO, ACC)                                                                                          \
    "add.u32 al, %1, " AO ";\n\tadd.u32 bl, %3, " BO ";\n\tmov.b64 da, {al, %2};\n\tmov.b64 db, {bl, %4};\n\t"       \
    "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, " ACC ";\n\t"
#define JL_SS_HEAD                                                                                                   \
    "{\n\t.reg .pred p, t, e;\n\t.reg .b32 al, bl;\n\t.reg .b64 da, db;\n\telect.sync _|e, 0xffffffff;\n\t"          \
    "setp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, %6, %6;\n\t"
#define JL_SS_ARGS                                                                                                   \
    "}" ::"r"(d), "r"((uint32_t)a), "r"((uint32_t)(a >> 32)), "r"((uint32_t)b), "r"((uint32_t)(b >> 32)), "r"(idesc), "r"(acc)
// K-major operands over 64 of the head dimensions (four steps inside one swizzle atom)
__device__ __forceinline__ void umma_ss_k64(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(JL_SS_HEAD JL_SS("0", "0", "p") JL_SS("2", "2", "t") JL_SS("4", "4", "t") JL_SS("6", "6", "t") JL_SS_ARGS : "memory");
}
// MN-major operands over 128 keys (eight steps of 16 rows of 128 bytes)
__device__ __forceinline__ void umma_ss_mn128(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(JL_SS_HEAD JL_SS("0", "0", "p") JL_SS("128", "128", "t") JL_SS("256", "256", "t") JL_SS("384", "384", "t")
                     JL_SS("512", "512", "t") JL_SS("640", "640", "t") JL_SS("768", "768", "t") JL_SS("896", "896", "t")
                         JL_SS_ARGS : "memory");
}
// D[tmem] += A B over 32 keys (two steps), A = weights in tensor memory, B = values
__device__ __forceinline__ void umma_ts_k32(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc)
{
    asm volatile(
        "{\n\t.reg .pred t, e;\n\t.reg .b32 ta, bl;\n\t.reg .b64 db;\n\telect.sync _|e, 0xffffffff;\n\t"
        "setp.eq.b32 t, %4, %4;\n\tmov.b64 db, {%2, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, t;\n\t"
        "add.u32 ta, %1, 8;\n\tadd.u32 bl, %2, 128;\n\tmov.b64 db, {bl, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %4, t;\n\t}"
        ::"r"(d), "r"(a), "r"((uint32_t)b), "r"((uint32_t)(b >> 32)), "r"(idesc) : "memory");
}
#undef JL_SS
#undef JL_SS_HEAD
#undef JL_SS_ARGS

// A pair of weights as two bf16 pairs whose sum has 16 bits of them: the upper half of
// the words, and what that leaves, rounded.  With weights of 8 bits the results of long
// caches were off by 2.4e-3 of their size (rms) where rounding the results themselves
// costs 1.6e-3.
__device__ __forceinline__ uint32_t split_weights(float a, float b, uint32_t& rest)
{
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    const float2 r = fma2(make_float2(__uint_as_float(x & 0xffff0000u), __uint_as_float(y & 0xffff0000u)),
                          make_float2(-1.f, -1.f), make_float2(a, b));
    rest = pack_bf16x2(r.x, r.y);
    return __byte_perm(x, y, 0x7632);
}

__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t mag16(uint32_t a) { return max(a & 0x7fffu, (a >> 16) & 0x7fffu); }

// Exponent of the power of two that brings a row's largest element into [2^13, 2^14)
// (at most 2^126, for subnormals); rows of zeros, or with infinities or NaN, stay.
__device__ __forceinline__ int row_exp(uint32_t mag)
{
    if (mag == 0u || mag >= 0x7f80u) return 0;
    return min(126, 140 - max((int)(mag >> 7), 1));
}

// Factor of a logit whose key row was scaled: that of its query row (cq) times the inverse
// key scale, formed first, since a raw logit times either alone can be outside fp32 where
// the logit is not.  (Too large a factor belongs to an infinite logit, or to a raw one of 0.)
__device__ __forceinline__ float logit_factor(float cq, float ks) { return fminf(cq * ks, 3.40282347e38f); }

// What every role sees.
template <class C>
struct Role {
    const PagedProblem& p;
    const Launch& ln;
    int warp, lane;
    __device__ __forceinline__ Role(const PagedProblem& p_, const Launch& ln_) : p(p_), ln(ln_)
    {
        warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
    }
    __device__ __forceinline__ volatile int* abort_flag() const { return reinterpret_cast<volatile int*>(smem_base() + C::SLOT + 4); }
    __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int code) const
    {
        // (the whole warp polls: one lane polling for the others took 10-40% longer, and
        // letting the hardware park the warp 10%)
        return tc::warp_wait(bar, parity, abort_flag(), ln.dev_error, ln.wait_cycles, code);
    }
    // unit k of the piece: wait until it is planned; afterwards each warp hands it back
    __device__ __forceinline__ bool unit_wait(int k, int code) const { return wait(&Bars<C>().dfull[k % UNITS], (k / UNITS) & 1, code); }
    __device__ __forceinline__ UnitPtr unit(int k) const { return reinterpret_cast<UnitDesc*>(smem_base() + C::DESC) + k % UNITS; }
    __device__ __forceinline__ void unit_done(int k) const
    {
        __syncwarp();
        if (lane == 0) mbar_arrive(&Bars<C>().dfree[k % UNITS]);
    }
    __device__ __forceinline__ volatile unsigned* note() const { return reinterpret_cast<volatile unsigned*>(smem_base() + C::NOTE); }
    __device__ __forceinline__ unsigned all_pages() const { return (1u << (KT >> min(p.page_shift, 7))) - 1; }
};

// Start of a CTA: barriers, tensor memory (warp 2), the plan of its piece.  Returns
// the tensor memory address.
template <class C, uint32_t TCOLS, class InitExtra>
__device__ __forceinline__ uint32_t start_cta(const Role<C>& ro, InitExtra init_extra)
{
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem_base() + C::SLOT);
    const int tid = threadIdx.x;
    if (tid == C::THREADS - 1) {  // (the first threads go on to the requests' lengths)
        Bars<C> bars;
        bars.init();
        init_extra();
        *ro.abort_flag() = *reinterpret_cast<volatile int*>(ro.ln.dev_error) != 0;  // an earlier wait ran out: no work
        fence_mbar_init();
    }
    for (int m = tid; m < C::DIM / 2; m += C::THREADS)
        reinterpret_cast<uint2*>(smem_base() + C::TURNS)[m] = make_uint2(ro.p.turns.hi[m], ro.p.turns.lo[m]);
    if (ro.warp == 2) {
        tmem_alloc(slot, TCOLS);
        tmem_relinquish();
        tc_fence_before();
    }
    // ends with a barrier of the CTA
    piece_plan<KT, C::ROWS, C::THREADS>(ro.p, ro.ln.min_items, reinterpret_cast<PiecePlan*>(smem_base() + C::PLAN),
                                        reinterpret_cast<long long*>(smem_base() + C::SCAN));
    tc_fence_after();
    return *slot;
}

// Producer of key tiles (warp 0) or value tiles (warp 3): the page numbers of a
// tile's rows, then one TMA box per page and 64 columns.  The value producer also
// clears what a request's last tile must not hold.
template <class C, bool isK>
__device__ __forceinline__ void produce(const Role<C>& ro, const CUtensorMap* tm)
{
    const PagedProblem& p = ro.p;
    const Launch& ln = ro.ln;
    unsigned char* const smem = smem_base();
    const Bars<C> bars;
    const int lane = ro.lane;
    constexpr int D = C::DIM;
    constexpr int NS = isK ? C::NSK : C::NSV;
    constexpr int NF = isK ? C::NKF : C::NSV;  // barriers of landed tiles
    uint64_t* full = isK ? bars.kfull : bars.vfull;
    uint64_t* empty = isK ? bars.kempty : bars.vempty;
    unsigned char* ring = smem + (isK ? C::K0 : C::V0);
    const int box = min(p.page_size, KT), gshift = min(p.page_shift, 7);
    const unsigned all_pages = ro.all_pages();
    int e = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
        if (!ro.unit_wait(k, isK ? 0x603 : 0x604)) break;
        UnitPtr un = ro.unit(k);
        if (un->rows == 0) break;
        const int* table = p.table + (size_t)un->b * p.max_pages;
        const int L = un->L, n = L + un->T, kvh = un->kvh;
        for (UnitItems it(un); it.left > 0; it.next(), ++e) {
            // lane x looks after rows [x box, (x + 1) box) of the tile
            const int j0 = it.tile * KT, row = j0 + lane * box;
            const bool want = lane * box < KT && row < n;
            int page = -1;
            if (want) {
                page = __ldg(table + (row >> p.page_shift));
                if ((unsigned)page >= (unsigned)p.num_pages) {
                    record_input(p.input_error, kBadPage);
                    page = -1;
                }
            }
            const int st = e % NS;
            if (e >= NS && !ro.wait(&empty[st], ((e / NS) - 1) & 1, isK ? 0x601 : 0x602)) { ok = false; break; }
            const unsigned have = __ballot_sync(0xffffffffu, page >= 0);
            const bool skip = isK && e == 0 && ln.inject == kInjectDecodeCopy;  // test hook: the first key tile is never loaded
            if (lane == 0) {
                if (isK) ro.note()[e % INFO] = have;
                if (!skip) {
                    if (have)
                        mbar_arrive_expect_tx(&full[e % NF], (uint32_t)(__popc(have) * box * D * 2));
                    else
                        mbar_arrive(&full[e % NF]);
                }
            }
            __syncwarp();
            if (page >= 0 && !skip) {
                unsigned char* dst = ring + st * C::TILE + lane * box * 128;
                const int y = row & (p.page_size - 1), z = page * p.Hkv + kvh;
#pragma unroll
                for (int a = 0; a < C::ATOMS; ++a) tma_load_3d(dst + a * C::ATOM_K, tm, a * 64, y, z, &full[e % NF]);
            }
            if (!isK && (j0 + KT > L || have != all_pages)) {
                // Value rows that do not exist count as zero: the page may hold anything
                // there, and a weight of 0 does not silence NaN.  A drafted row's own
                // infinities and NaN are cleared as well (nodes beside it must not see
                // them) and noted for the nodes that do attend it.
                if (!ro.wait(&full[e % NF], (e / NF) & 1, 0x605)) {
                    ++e;  // its copy is in flight
                    ok = false;
                    break;
                }
                unsigned char* vt = ring + st * C::TILE;
                const int first = have == all_pages ? max(0, L - j0) : 0;
                for (int r = first + lane; r < KT; r += 32) {
                    const int j = j0 + r;
                    const bool there = j < n && ((have >> (r >> gshift)) & 1);
                    if (there && j < L) continue;
                    bool hit = false;
#pragma unroll 4
                    for (int x = 0; x < D / 8; ++x) {
                        uint4* v = reinterpret_cast<uint4*>(vt + tc::sw128_off<KT>(r, x));
                        if (!there) {
                            *v = make_uint4(0u, 0u, 0u, 0u);
                            continue;
                        }
                        uint4 w = *v;
                        uint32_t* y = &w.x;
                        bool any = false;
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            if ((y[u] & 0x7f80u) == 0x7f80u) { y[u] &= 0xffff0000u; any = true; }
                            if ((y[u] & 0x7f800000u) == 0x7f800000u) { y[u] &= 0xffffu; any = true; }
                        }
                        if (any) *v = w;
                        hit |= any;
                    }
                    if (hit) atomicOr(const_cast<unsigned long long*>(&un->bad), 1ull << (j - L));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.vfix[st]);
            }
        }
        ro.unit_done(k);
    }
    // the copies in flight land before the CTA ends
    for (int x = max(0, e - NS); x < e; ++x)
        if (!(isK && x == 0 && ln.inject == kInjectDecodeCopy)) mbar_wait(&full[x % NF], (x / NF) & 1);
}

// Planner (one thread of warp 2): the units of this CTA's piece, a few ahead.
template <class C>
__device__ __forceinline__ void plan_units(const Role<C>& ro)
{
    const PagedProblem& p = ro.p;
    const PiecePlan* plan = reinterpret_cast<const PiecePlan*>(smem_base() + C::PLAN);
    const Bars<C> bars;
    if (ro.lane == 0) {
        long long cur = plan->start, base = plan->base;
        clear_cut(p);
        const long long end = *ro.abort_flag() ? cur : plan->end;
        int b = plan->b, k = 0;
        SeqPlan s = plan->first;
        for (;; ++k) {
            UnitDesc u;
            u.rows = 0;
            u.bad = 0;
            if (cur < end) {
                long long cnt = (long long)s.items * s.row_tiles * p.Hkv;
                while (cur >= base + cnt) {
                    base += cnt;
                    ++b;
                    s = seq_plan<KT, C::ROWS>(p, b, false);
                    cnt = (long long)s.items * s.row_tiles * p.Hkv;
                }
                int unit;
                div_items(cur - base, s.items, &unit, &u.i0);
                u.i1 = (int)min((long long)s.items, u.i0 + (end - cur));
                u.kvh = unit / s.row_tiles;
                u.r0 = (unit % s.row_tiles) * C::ROWS;
                u.rows = min(C::ROWS, s.T * p.group - u.r0);
                u.L = s.L;
                u.T = s.T;
                u.n0 = s.n0;
                u.b = b;
                u.gmin = s.gmin;
                u.ng = s.ng;
                u.nR = s.nR;
                u.kE0 = s.kE0;
                u.w0 = s.w0;
                u.items = s.items;
            }
            if (k >= UNITS && !tc::wait_or_abort(&bars.dfree[k % UNITS], ((k / UNITS) - 1) & 1, ro.abort_flag(), ro.ln.dev_error, ro.ln.wait_cycles, 0x641))
                break;
            reinterpret_cast<UnitDesc*>(smem_base() + C::DESC)[k % UNITS] = u;
            mbar_arrive(&bars.dfull[k % UNITS]);
            if (u.rows == 0) break;
            if (u.i0 == 0 && u.i1 < s.items) note_cut(p, s, plan->per, cur, u.kvh, u.r0, u.rows);
            cur += u.i1 - u.i0;
        }
    }
    __syncwarp();
}

// Rotation (C::ROTALL threads from thread 128 on).  Per unit: the tree, positions and
// query scales.  Per phase: the queries rotated into shared memory.  Per tile: the
// keys rotated in place.
template <class C>
__device__ __forceinline__ void rotate_keys(const Role<C>& ro)
{
    const PagedProblem& p = ro.p;
    unsigned char* const smem = smem_base();
    const Bars<C> bars;
    const int lane = ro.lane;
    constexpr int D = C::DIM, H = D / 2, CH = D / 16, NSK = C::NSK;
    float* ksc = reinterpret_cast<float*>(smem + C::KSC);
    const int t = (int)threadIdx.x - 128, rt = t & (C::ROT - 1);  // thread of the role, of the tile
    const int group = C::ALT ? t >> 7 : 0;
    constexpr int RPT = KT * CH / C::ROT;          // rows per thread of a tile: 128 rows x CH chunk pairs
    const int c = t % CH, row0 = (rt / CH) * RPT;
    const uint4* turns = reinterpret_cast<const uint4*>(smem + C::TURNS) + c * 4;  // the thread's 8 frequencies
    float2 stc[4], sts[4];                         // cos, sin of one position step, as frequency pairs
    struct Angles {
        float2 cs[4], sn[4];  // cos, sin of the 8 frequencies, as pairs
    };
    auto angles = [&](uint32_t f, Angles& a) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint4 w2 = turns[u];
            rope_cs_fast(f, w2.x, w2.y, a.cs[u].x, a.sn[u].x);
            rope_cs_fast(f, w2.z, w2.w, a.cs[u].y, a.sn[u].y);
        }
    };
    {
        Angles one;
        angles(1u, one);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            stc[u] = one.cs[u];
            sts[u] = one.sn[u];
        }
    }
    // 8 pairs (lo.x holds dimensions 0, 1 of the chunk, hi.x their partners, ...)
    // turned by (cs, sn), as fp16
    auto turn = [&](uint4& lo, uint4& hi, const Angles& by) {
        uint32_t* a = &lo.x;
        uint32_t* b = &hi.x;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float2 x = make_float2(bf16_lo(a[u]), bf16_hi(a[u])), y = make_float2(bf16_lo(b[u]), bf16_hi(b[u]));
            const float2 ny = make_float2(__uint_as_float((b[u] << 16) + 0x80000000u),
                                          __uint_as_float((b[u] & 0xffff0000u) ^ 0x80000000u));
            const float2 r0 = fma2(ny, by.sn[u], mul2(x, by.cs[u])), r1 = fma2(y, by.cs[u], mul2(x, by.sn[u]));
            a[u] = pack_f16x2(r0.x, r0.y);
            b[u] = pack_f16x2(r1.x, r1.y);
        }
    };
    auto absmax8 = [](const uint4& a, const uint4& b) {
        return absmax2(absmax2(absmax2(a.x, a.y), absmax2(a.z, a.w)), absmax2(absmax2(b.x, b.y), absmax2(b.z, b.w)));
    };
    auto sum8 = [](const uint4& a) {
        return fabsf(bf16_lo(a.x)) + fabsf(bf16_hi(a.x)) + fabsf(bf16_lo(a.y)) + fabsf(bf16_hi(a.y)) + fabsf(bf16_lo(a.z)) +
               fabsf(bf16_hi(a.z)) + fabsf(bf16_lo(a.w)) + fabsf(bf16_hi(a.w));
    };
    auto scale8 = [](uint4& a, float sc) {  // exact: a power of two (elements far below the row's largest may vanish)
        a.x = pack_bf16x2(bf16_lo(a.x) * sc, bf16_hi(a.x) * sc);
        a.y = pack_bf16x2(bf16_lo(a.y) * sc, bf16_hi(a.y) * sc);
        a.z = pack_bf16x2(bf16_lo(a.z) * sc, bf16_hi(a.z) * sc);
        a.w = pack_bf16x2(bf16_lo(a.w) * sc, bf16_hi(a.w) * sc);
    };
    int* par = reinterpret_cast<int*>(smem + C::PAR);
    unsigned long long* nanc = reinterpret_cast<unsigned long long*>(par + kMaxNodes);
    int e = 0, nu = 0;
    // A wait that runs out in one warp must not leave the others at a barrier:
    // the warps meet once per unit (and once after the last) and stop together
    // if any of them gave up.
    bool ok = true, agreed = false;
    for (; ok; ++nu) {
        ok = ro.unit_wait(nu, 0x626);
        UnitPtr ud = ro.unit(nu);
        if (ok && ud->rows == 0) break;
        unsigned char* un = smem + C::UNIT + (nu & 1) * C::UBYTES;
        int* depth = reinterpret_cast<int*>(un + C::U_DEPTH);
        int* lim0 = reinterpret_cast<int*>(un + C::U_LIM);
        int* qG = reinterpret_cast<int*>(un + C::U_QG);
        float* cq = reinterpret_cast<float*>(un + C::U_CQ);
        unsigned long long* canc = reinterpret_cast<unsigned long long*>(un + C::U_ANC);
        int* big = reinterpret_cast<int*>(un + C::U_BIG);
        // the softmax is done with unit nu - 2, the tensor cores with the queries of
        // unit nu - 1 (known to the warps that rotated item e - 1, and through the
        // barrier to the others)
        ok = ok && (nu < 2 || ro.wait(&bars.ufree[nu & 1], ((nu >> 1) - 1) & 1, 0x621)) &&
             (e == 0 || ro.wait(&bars.kempty[(e - 1) % NSK], ((e - 1) / NSK) & 1, 0x622));
        if ((agreed = named_or(1, C::ROTALL, !ok))) break;
        const int L = ud->L, T = ud->T, n = L + T, rows = ud->rows, r0 = ud->r0, kvh = ud->kvh, n0 = ud->n0;
        // up to ROTALL / CH rows: a thread holds one chunk of one query for the whole unit,
        // on its way while the tree is read
        constexpr bool ONE = C::ROWS * CH <= C::ROTALL;
        const int own_row = ONE ? t / CH : 0, own_node = ONE ? min((r0 + own_row) / p.group, T - 1) : 0;
        uint4 own_lo = make_uint4(0u, 0u, 0u, 0u), own_hi = own_lo;
        if (ONE && own_row < rows) {
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) +
                                     ((size_t)(n0 + own_node) * p.Hq + kvh * p.group + (r0 + own_row) % p.group) * D + c * 8;
            own_lo = *reinterpret_cast<const uint4*>(q);
            own_hi = *reinterpret_cast<const uint4*>(q + H);
        }
        if (t < T) {
            int x = t - 1;
            if (p.parents) {
                x = p.parents[n0 + t];
                if (x < -1 || x >= t) {
                    record_input(p.input_error, kBadParent);
                    x = -1;
                }
            }
            par[t] = x;
        }
        if (t == 0) *big = 0;
        named_sync(1, C::ROTALL);
        if (t < T) {
            unsigned long long m = (2ull << t) - 1;
            if (p.parents) {
                m = 0;
                for (int x = t; x >= 0; x = par[x]) m |= 1ull << x;
            }
            nanc[t] = m;
            depth[t] = __popcll(m) - 1;
        }
        named_sync(1, C::ROTALL);
        // The unit's queries turned for the phase of group size g, as fp16.  The first time
        // also the rows' notes: each query is multiplied by a power of two that brings its
        // largest element into [2^13, 2^14), its logits by the inverse.
        //
        // One chunk of one query, by CH lanes that share the row:
        auto query = [&](bool live, int node, int row, uint4 lo, uint4 hi, const Angles& by, bool setup) {
            uint32_t mx = mag16(absmax8(lo, hi));
#pragma unroll
            for (int o = 1; o < CH; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            // (cq stays a normal number; logits of smaller queries are below 2^-4)
            const int ex = min(row_exp(mx), (int)(__float_as_uint(p.scale_log2) >> 23) - 1);
            const float sc = tc::pow2i(ex);
            if (setup) {
                float l1 = sum8(lo) + sum8(hi);
#pragma unroll
                for (int o = 1; o < CH; o <<= 1) l1 += __shfl_xor_sync(0xffffffffu, l1, o);
                if (c == 0 && live) {
                    const int pos = L + depth[node];
                    lim0[row] = pos - ud->w0;
                    qG[row] = pos / p.w_pre + 1;
                    canc[row] = nanc[node];
                    // a normal number: -inf times it stays -inf
                    cq[row] = fminf(fmaxf(tc::pow2i(-ex) * p.scale_log2, 1.17549435e-38f), 3.40282347e38f);
                    // keys rounded to fp16 as they are err by up to 2^-25 where fp16 is
                    // subnormal; with an L1 norm this large that could reach 2^-11 of a logit
                    if (!(l1 * p.scale_log2 * 1.4142136f <= 16384.f)) *big = 1;
                }
            }
            if (live) {
                scale8(lo, sc);
                scale8(hi, sc);
                turn(lo, hi, by);
                *reinterpret_cast<uint4*>(smem + C::Q0 + C::q_off(row, c)) = lo;
                *reinterpret_cast<uint4*>(smem + C::Q0 + C::q_off(row, c + CH)) = hi;
            }
        };
        auto load_query = [&](int node, int h, uint4& lo, uint4& hi) {
            const __nv_bfloat16* q =
                static_cast<const __nv_bfloat16*>(p.q) + ((size_t)(n0 + node) * p.Hq + kvh * p.group + h) * D + c * 8;
            lo = *reinterpret_cast<const uint4*>(q);
            hi = *reinterpret_cast<const uint4*>(q + H);
        };
        // More rows than that: a task is a chunk of `span` heads of one node, which share
        // their angles.
        const int node0 = r0 / p.group, nodes = (r0 + rows - 1) / p.group - node0 + 1;
        const int span = min(p.group, (rows * CH + C::ROTALL - 1) / C::ROTALL);
        const int spans = (p.group + span - 1) / span;
        auto queries = [&](int g, bool setup) {
            if (ONE) {
                Angles by;
                angles((uint32_t)(L + depth[own_node]) / (uint32_t)max(g, 1), by);
                query(own_row < rows, own_node, own_row, own_lo, own_hi, by, setup);
            } else {
                const int tasks = nodes * spans * CH, end = (tasks + 31) / 32 * 32;  // whole warps
#pragma unroll 1
                for (int x = t; x < end; x += C::ROTALL) {  // CH divides the thread count: chunk x % CH = c
                    const int y = x / CH, node = min(node0 + y / spans, T - 1), h0 = (y % spans) * span;
                    Angles by;
                    angles((uint32_t)(L + depth[node]) / (uint32_t)max(g, 1), by);
#pragma unroll 1
                    for (int h = h0; h < h0 + span; ++h) {
                        const int row = node * p.group + h - r0;
                        const bool live = x < tasks && h < p.group && row >= 0 && row < rows;
                        uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
                        if (live) load_query(node, h, lo, hi);
                        query(live, node, row, lo, hi, by, setup);
                    }
                }
            }
            if (setup) {
                // Rows without a query: zeros, no drafted row attended.  (What shared memory held
                // before must not decide whether the softmax moves its references: those of the
                // other rows would move with them, and results change in their last bit.)
                for (int row = rows + t; row < C::ROWS; row += C::ROTALL) {
                    lim0[row] = qG[row] = 0;
                    canc[row] = 0ull;
                    cq[row] = 1.f;
                }
                for (int x = rows * 2 * CH + t; x < C::ROWS * 2 * CH; x += C::ROTALL)
                    *reinterpret_cast<uint4*>(smem + C::Q0 + C::q_off(x / (2 * CH), x % (2 * CH))) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.qready);
        };
        UnitItems it(ud);
        int gcur = it.g;
        queries(gcur, true);
        named_sync(1, C::ROTALL);
        if (lane == 0) mbar_arrive(&bars.uready[nu & 1]);
        const bool always = *big != 0;
        uint32_t dm = 0, ds1 = 0, ds2 = 0;  // division by the group size by multiply-shift
        auto set_divisor = [&](int g) {
            const uint32_t dv = max(g, 1);
            const uint32_t lg = 32 - __clz(dv - 1);  // ceil(log2 dv); 0 for 1
            dm = (uint32_t)(((((uint64_t)1 << 32) * (((uint64_t)1 << lg) - dv)) / dv) + 1);
            ds1 = min(lg, 1u);
            ds2 = lg > 1 ? lg - 1 : 0;
        };
        set_divisor(gcur);
        for (; it.left > 0; it.next(), ++e) {
            if (it.g != gcur) {
                // the next phase; the tensor cores are done with the queries of the last
                // (only the warps that rotated item e - 1 know that the wait is for its phase:
                // the others follow through the barrier)
                ok = ro.wait(&bars.kempty[(e - 1) % NSK], ((e - 1) / NSK) & 1, 0x623);
                if ((agreed = named_or(1, C::ROTALL, !ok))) {
                    ok = false;
                    break;
                }
                gcur = it.g;
                set_divisor(gcur);
                queries(gcur, false);
            }
            if (C::ALT && (e & 1) != group) continue;
            const int st = e % NSK, j0 = it.tile * KT;
            unsigned char* kt = smem + C::K0 + st * C::TILE;
            const bool drafted = j0 + KT > L;
            auto over_g = [&](uint32_t pos) {
                const uint32_t t1 = __umulhi(dm, pos);
                return (t1 + ((pos - t1) >> ds1)) >> ds2;
            };
            // Keys are rounded to fp16 as they are, unless one of the warp's is too large
            // for it (0x4700: 2^15), or the query makes small ones count: then every row is
            // first scaled by its own power of two.  `top` covers the rows at hand.
            unsigned scaled = 0;
            auto too_large = [&](uint32_t top) { return __any_sync(0xffffffffu, always || mag16(top) >= 0x4700u); };
            auto scale_row = [&](uint4& lo, uint4& hi) {
                uint32_t m = mag16(absmax8(lo, hi));
#pragma unroll
                for (int o = 1; o < CH; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                const int ex = row_exp(m);
                scale8(lo, tc::pow2i(ex));
                scale8(hi, tc::pow2i(ex));
                scaled = 1;
                return tc::pow2i(-ex);
            };
            float* kscale = ksc + (e % INFO) * KT;
            Angles by;
            if (!drafted) {
                // committed rows: the turned position of row j is floor(j / g); from row to
                // row it stays or steps by one, and the angles follow by angle addition.
                // (The loop body is kept small: five roles share the instruction cache, and
                // with four rows per turn the 128K batch took 1130 us instead of 810.)
                uint32_t f = over_g((uint32_t)(j0 + row0));
                angles(f, by);
                if (!ro.wait(&bars.kfull[e % C::NKF], (e / C::NKF) & 1, 0x624)) { ok = false; break; }
                auto advance = [&](int r) {
                    const uint32_t fn = over_g((uint32_t)(j0 + r));
                    if (fn != f) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float2 nc = fma2(make_float2(-by.sn[u].x, -by.sn[u].y), sts[u], mul2(by.cs[u], stc[u]));
                            by.sn[u] = fma2(by.cs[u], sts[u], mul2(by.sn[u], stc[u]));
                            by.cs[u] = nc;
                        }
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
                    float2 ks = make_float2(1.f, 1.f);
                    if (too_large(absmax2(absmax8(a0, b0), absmax8(a1, b1)))) {
                        ks.x = scale_row(a0, b0);
                        ks.y = scale_row(a1, b1);
                    }
                    if (c == 0) *reinterpret_cast<float2*>(kscale + r) = ks;
                    if (x > 0) advance(r);
                    turn(a0, b0, by);
                    *pa = a0;
                    *pb = b0;
                    advance(r + 1);
                    turn(a1, b1, by);
                    *pc = a1;
                    *pd = b1;
                }
            } else {
                // a request's last tiles: drafted rows sit at their depths.  Rows past the end
                // are masked, and zeroed: large numbers there would have their neighbours
                // scaled, and so rounded in another way.
                if (!ro.wait(&bars.kfull[e % C::NKF], (e / C::NKF) & 1, 0x624)) { ok = false; break; }
#pragma unroll 1
                for (int x = 0; x < RPT; ++x) {
                    const int r = row0 + x, j = j0 + r;
                    angles(over_g(j < L ? (uint32_t)j : j < n ? (uint32_t)(L + depth[j - L]) : 0u), by);
                    uint4* pa = reinterpret_cast<uint4*>(kt + tc::sw128_off<KT>(r, c));
                    uint4* pb = reinterpret_cast<uint4*>(kt + tc::sw128_off<KT>(r, c + CH));
                    uint4 a = *pa, b = *pb;
                    if (j >= n) a = b = make_uint4(0u, 0u, 0u, 0u);
                    float ks = 1.f;
                    if (too_large(absmax8(a, b))) ks = scale_row(a, b);
                    if (c == 0) kscale[r] = ks;
                    turn(a, b, by);
                    *pa = a;
                    *pb = b;
                }
            }
            if (lane == 0) reinterpret_cast<volatile unsigned*>(smem + C::SCALED)[(e % INFO) * 8 + (rt >> 5)] = scaled;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.kready[st]);
        }
        ro.unit_done(nu);
    }
    if (!agreed) named_or(1, C::ROTALL, !ok);
}

}  // namespace ptc
}  // namespace jl
