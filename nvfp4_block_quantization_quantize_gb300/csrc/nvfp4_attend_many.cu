// nvfp4_attend_many.cu -- attention of many queries a sequence over a paged NVFP4 cache: the
// sequences of nvfp4_cache_attention with more rows than the warp-level kernel is for (is_many).
//
// The rows are a sequence's queries times the heads that share a KV head; two tiles of
// 128 rows share each block of 128 keys.  4 D operations a row and key: bound by the tensor
// cores (tcgen05, f16, fp32 sums in tensor memory), with 256 rows' softmax and the decoding of a block beside them.
//   - Producers (a warpgroup for keys, one for values) load the next block's codes into registers while they decode
//     the present one to f16 in shared memory, exactly (q * dec(s)); keys and values lie alike, 64 elements of a
//     token to 128 swizzled bytes: K-major for S = Q K^T, MN-major for O += P V.
//   - One warp issues the products: S of tile A, S of B, then for each block O of a tile and its next S.
//     While one tile's softmax runs the other's products do.
//   - A softmax warpgroup a tile, a thread a row: S out of tensor memory, weights back as f16 over S,
//     which P V reads from there.  Weights are made by a reference as it stands: while a block's sum is at
//     most 65504 each of them fits f16, and no maximum is looked for.  Else, or where so little is left of
//     them that f16 would lose bits, the reference is moved by the sum, O, in tensor memory too, is rescaled
//     and the block's weights are made again.
// Queries enter as f16 scaled by a power of two for each row, as in the other kernel.
// Measured: the last 2048 queries of 2 sequences of 16384 keys, 32 heads of 128 over 8, causal: 702 us, 1.47 PFLOP/s (of 1.92 of a large
// product; the warp-level kernel's way took 4.9 ms).  A maximum looked for in each block took 1.78 ms, one warpgroup
// decoding keys and values 0.81 ms.  What is left is shared: without the softmax's arithmetic 713 of then 771 us, without the
// decoding 685, with a quarter of the products 662, with none of the three 361.
// Equal runs of blocks for each CTA, whatever the sequences; cut groups are joined by k_join.  A group costs 9 us besides
// its blocks (1.5 us each, a masked one 4): queries, first copies and the end are not all behind another's products.
#include "nvfp4_attend.cuh"

namespace nvfp4 {
namespace {

constexpr int kRows = 256;                                // of a group: two tiles of 128
constexpr int kKeys = 128;                                // of a block
constexpr int kThreadsMany = 640;                         // warpgroups: products, softmax A, softmax B, keys, values
constexpr int kLaunchRegisters = 96;                      // of a thread

// registers of a thread after they are shared out anew
constexpr int kSoftmaxRegisters = 128, kProducerRegisters = 80, kProductRegisters = 64;
static_assert(128 * (2 * kSoftmaxRegisters + 2 * kProducerRegisters + kProductRegisters) <= kThreadsMany * kLaunchRegisters,
              "no more than were launched");

enum Bar { kQFull, kQEmpty, kKFull, kKEmpty = kKFull + 2, kVFull = kKEmpty + 2, kVEmpty = kVFull + 2, kSFull = kVEmpty + 2,
           kPFull = kSFull + 2, kOFull = kPFull + 2, kRaw = kOFull + 2, kBars = kRaw + 2 };

// ---- tcgen05 --------------------------------------------------------------------------------------
// .kind::f16: f16 operands, fp32 sums; B K-major or MN-major
__device__ __forceinline__ uint32_t idesc_f16(int M, int N, bool b_mn) {
    return 1u << 4 | (b_mn ? 1u << 16 : 0u) | static_cast<uint32_t>(N >> 3) << 17 | static_cast<uint32_t>(M >> 4) << 24;
}

// A matrix descriptor's upper word is the same for all operands of a kind; the lower is an address (in 16 bytes) and the
// step between pieces along the other way.  Steps are added where the product is issued: as values of their own they would
// fill the registers.
constexpr uint32_t kDescUpper = 1024 >> 4 | 1u << 14 | 2u << 29;      // 8 rows of 128 swizzled bytes apart (smem_desc)

template <int STEP_A, int STEP_B>
__device__ __forceinline__ void mma_ss(uint32_t el, uint32_t d, uint32_t da, uint32_t db, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 x, y;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "add.u32 x, %1, %6;\n\t"
        "add.u32 y, %2, %7;\n\t"
        "mov.b64 da, {x, %8};\n\t"
        "mov.b64 db, {y, %8};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(da), "r"(db), "r"(idesc), "r"(acc), "r"(el), "n"(STEP_A), "n"(STEP_B), "n"(kDescUpper)
        : "memory");
}

// A from tensor memory
template <int STEP_B>
__device__ __forceinline__ void mma_ts(uint32_t el, uint32_t d, uint32_t ta, uint32_t db, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 y;\n\t.reg .b64 db;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "add.u32 y, %2, %6;\n\t"
        "mov.b64 db, {y, %7};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(ta), "r"(db), "r"(idesc), "r"(acc), "r"(el), "n"(STEP_B), "n"(kDescUpper)
        : "memory");
}

// 32 columns of this thread's row
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}

__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// until loads are in; v: what they gave, so that nothing uses it before
__device__ __forceinline__ void tmem_wait_load(uint32_t* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]),
                   "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]),
                   "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// 16 bytes of codes and 2 of scales, zeros where not wanted (without a branch)
__device__ __forceinline__ void load_if(bool wanted, const uint8_t* codes, const uint8_t* scales, uint4& w, uint32_t& sc) {
    uint16_t s;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %7, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\tmov.b16 %4, 0;\n\t"
        "@p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%5];\n\t"
        "@p ld.global.nc.b16 %4, [%6];\n\t}"
        : "=&r"(w.x), "=&r"(w.y), "=&r"(w.z), "=&r"(w.w), "=&h"(s)
        : "l"(codes), "l"(scales), "r"(static_cast<int>(wanted)));
    sc = s;
}

template <int N>
__device__ __forceinline__ void registers_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void registers_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ bool done(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok;
}

// A warp's wait; it ends too when another one has run out.  False then, for all lanes.
__device__ __forceinline__ bool long_wait(uint64_t* bar, uint32_t parity, volatile int* lost) {
    for (long it = 0; it < kWaitLimit; ++it) {
        if (__all_sync(kFullMask, done(bar, parity))) return true;
        if ((it & 15) == 15 && __any_sync(kFullMask, *lost)) return false;
    }
    *lost = 1;
    return false;
}

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* lost) {
    return __all_sync(kFullMask, done(bar, parity)) || long_wait(bar, parity, lost);
}

template <int N>
struct Constant {
    static constexpr int value = N;
};

template <int N, class F>
__device__ __forceinline__ void unrolled(F f) {           // f(0) .. f(N - 1), each with its constant
    if constexpr (N > 0) {
        unrolled<N - 1>(f);
        f(Constant<N - 1>());
    }
}

// The work of a sequence, in keys that its groups of 256 rows are to look at: w0 + rt * step a group of row tile rt (the
// first kGroupKeys for what it costs besides: a prompt of 8192 queries, 32 heads of 128 over 8, took 804 us with 256, 589 with
// 512, 478 with 768, 465 with 1024; of 2048 91, 85, 83, 85).  With a causal mask the row tiles look at more and more; that they look at whole
// blocks, and a window cuts off the first keys, is not counted.
constexpr int kGroupKeys = 768;
constexpr int kMinKeys = 512;                             // a CTA's run is not made shorter

struct Load {
    int64_t w0;
    int rts, step;

    __device__ __forceinline__ Load(const AttendArgs& a, const Seq& s) {
        const int G = a.Hq / a.cache.Hkv, queries = (kRows + G - 1) / G;
        rts = s.runs / a.cache.Hkv;
        step = a.causal && !a.window ? queries : 0;
        w0 = kGroupKeys + (step ? max(s.len - s.n, 0) + step : a.window ? min(s.len, a.window + queries) : s.len);
    }
    __device__ __forceinline__ int64_t before(int64_t rt) const { return rt * w0 + rt * (rt - 1) / 2 * step; }
    __device__ __forceinline__ int64_t of(int rt) const { return w0 + static_cast<int64_t>(rt) * step; }
};

struct Keys {
    __device__ __forceinline__ static int64_t share(const AttendArgs& a, int64_t b) {
        const Load l(a, sequence<kRows>(a, b));
        return l.before(l.rts) * a.cache.Hkv;
    }
};

// A place in the work: before block blk of a group (b: a.B at the end of all), whose share of the work ends at key `until`.
struct Spot {
    int64_t b, until;
    int rt, h, blk;

    __device__ __forceinline__ bool group_of(const Spot& o) const { return b == o.b && rt == o.rt && h == o.h; }
};

// 256 rows of a sequence's KV head, and its blocks of keys
struct Item {
    Seq s;
    int rows, blocks, j0;             // the first key of its first block
    int first, last;                  // queries of its first and last row

    __device__ __forceinline__ Item(const AttendArgs& a, const Seq& seq, int rt) : s(seq) {
        const int G = a.Hq / a.cache.Hkv;
        rows = min(kRows, s.n * G - rt * kRows);
        int head;
        split_row(s.n, G, rt * kRows, &first, &head);
        split_row(s.n, G, rt * kRows + rows - 1, &last, &head);
        const int pos0 = s.len - s.n;
        const int lo = a.window > 0 ? max(0, pos0 + first - a.window + 1) : 0;
        const int hi = a.causal ? min(s.len, max(pos0 + last + 1, 0)) : s.len;
        j0 = lo / 16 * 16;
        blocks = hi > j0 ? (hi - j0 + kKeys - 1) / kKeys : 0;
    }
};

// where the run that would start at key x of all does.  Every lane of a warp calls it.
__device__ __forceinline__ Spot spot_of(const AttendArgs& a, const Shares<Keys>& shares, int64_t x) {
    Spot p{a.B, 0, 0, 0, 0};
    if (x >= shares.total) return p;
    int64_t before;
    shares.find(a, x, &p.b, &before);
    const Seq s = sequence<kRows>(a, p.b);
    const Load l(a, s);
    x -= before;
    int lo = 0, hi = l.rts - 1;                           // the last row tile that does not start after x
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (l.before(mid) * a.cache.Hkv <= x) lo = mid;
        else hi = mid - 1;
    }
    x -= l.before(lo) * a.cache.Hkv;
    const int64_t w = l.of(lo);
    p.rt = lo;
    p.h = static_cast<int>(quotient(x, w));
    p.until = before + l.before(lo) * a.cache.Hkv + (p.h + 1) * w;
    p.blk = static_cast<int>(quotient((x - p.h * w) * Item(a, s, lo).blocks, w));
    return p;
}

// CTAs that take part
__device__ __forceinline__ int64_t runs_of(int64_t keys, int64_t ctas) {
    const int64_t most = (keys + kMinKeys - 1) / kMinKeys;
    return most < ctas ? most : ctas;
}

// A CTA's run of parts of groups, as a warp walks along it (in shared memory; one lane walks).
struct Run {
    Spot at;
    Seq s;
    bool known, first, more;          // s is at.b's; nothing was done yet; there is a part: blocks at.blk .. to of at's group

    __device__ __forceinline__ void look(const AttendArgs& a, const Spot& end) {
        while (true) {
            // (a run that ends where it starts, amid a group, is an empty part of it)
            more = at.b < a.B && (!at.group_of(end) || (first ? end.blk > 0 : at.blk < end.blk));
            if (!more) return;
            if (!known) s = sequence<kRows>(a, at.b);
            known = true;
            if (s.runs > 0) return;
            ++at.b, at.rt = at.h = at.blk = 0, known = first = false;
        }
    }
    __device__ __forceinline__ void start(const AttendArgs& a, const Spot& from, const Spot& end) {
        at = from, known = false, first = true;
        look(a, end);
    }
    __device__ __forceinline__ void step(const AttendArgs& a, const Spot& end) {
        first = false;
        at.blk = at.group_of(end) ? end.blk : 0;
        if (!at.group_of(end) && ++at.h == a.cache.Hkv) {
            at.h = 0;
            if (++at.rt == s.runs / a.cache.Hkv) at.rt = 0, ++at.b, known = false;
        }
        look(a, end);
    }
    __device__ __forceinline__ int to(const Item& it, const Spot& end) const { return at.group_of(end) ? end.blk : it.blocks; }
};

template <int D>
struct Many {
    static constexpr int half = kKeys * 128;              // 64 elements of 128 tokens
    static constexpr int tile = D / 64 * half;            // Q of a tile, K or V of a block
    static constexpr int stages = 2;                      // blocks of K, and of V
    static constexpr int q = 0, k = 2 * tile, v = k + stages * tile;
    static constexpr int stage = v + stages * tile;       // of rows on their way out: [8 softmax warps][32 rows][128 bytes]
    static constexpr int factor = stage + 8 * 32 * 128;   // [256] fp32
    static constexpr int bars = factor + kRows * 4;
    static constexpr int spots = bars + 256;              // where the runs of the CTA before, of this and the next start
    static constexpr int runs = spots + 3 * sizeof(Spot); // of each warp
    static constexpr int bytes = runs + kThreadsMany / 32 * sizeof(Run);
    // tensor memory: S (and P over it) of A and B, O of A and B
    static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
    static constexpr int s_col = 0, o_col = 2 * kKeys;
    static constexpr int cols = 512;
    static_assert(2 * kKeys + 2 * D <= cols, "O of two tiles fits");
};

// bits from .. to - 1 of 32
__device__ __forceinline__ uint32_t columns(int from, int to) {
    const uint32_t below = to >= 32 ? ~0u : to <= 0 ? 0u : (1u << to) - 1u;
    return from >= 32 ? 0u : from <= 0 ? below : below & ~((1u << from) - 1u);
}

// A row's reference stands kBaseMany below the largest logit of its first block.  It is raised where a block's weights add up to
// more than kMostSum (each of them fits f16), so that they add up to 2^kUpSum, and lowered where they add up to less than kLeastSum,
// so that they add up to 2^kDownSum: half a step of f16's small values, 2^-25, of 128 weights is then at most 2^-9 of a
// block's sum, and 2^-29 of the largest weight of a block that sets or raises the reference.  It is lowered by at most kDrop, and
// where the denominator is below kFar, so that sums stay far inside fp32.  A call of 2 x 2048 queries on 16384 keys, logits spread by
// 3 nats / by 6 / by 12: 717, 832 and 1040 us with a base of 0, raised to the largest logit and never lowered; 726, 1134 and 1406
// lowered to it too; by sums 714, 932 and 1117 (a base of 2 716, 6 731, 8 778; lowered below 2^-12 709, 879 and 1109).
constexpr float kBaseMany = 4.0f, kMostSum = 65504.0f, kLeastSum = 0.001953125f, kUpSum = 12.0f, kDownSum = -2.0f;
constexpr float kDrop = 24.0f, kFar = 16777216.0f;

// Whether the reference is to be moved for a block's sum: the sum is outside [kLeastSum, kMostSum], and l, where the sum is low, below
// kFar.  (Positive floats compare as their bits; l stays below 2^49, since it is below kFar when it is scaled up by 2^kDrop.)
__device__ __forceinline__ bool misplaced(float sum, float l) {
    const uint32_t x = __float_as_uint(fmaxf(sum, mul_rn(l, kLeastSum / kFar)));
    return x - __float_as_uint(kLeastSum) > __float_as_uint(kMostSum) - __float_as_uint(kLeastSum);
}

// The keys of a block that a row sees: from lo to hi, relative to the block, of tiles that have a page.
struct Seen {
    int lo, hi;
    uint32_t have;

    __device__ __forceinline__ uint32_t of(int q) const {  // columns 32 q ..
        return columns(lo - 32 * q, hi - 32 * q) & ((have >> 2 * q & 1 ? 0xFFFFu : 0u) | (have >> 2 * q & 2 ? 0xFFFF0000u : 0u));
    }
};

// The largest logit of a row's block (kNone if it sees none).
__device__ __forceinline__ float largest(Seen seen, uint32_t s_at) {
    float top = kNone;
#pragma unroll 1
    for (int q = 0; q < kKeys / 32; ++q) {
        uint32_t v[32];
        __syncwarp();
        tmem_load32(s_at + 32 * q, v);
        tmem_wait_load(v);
        const uint32_t see = seen.of(q);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            top = max_nd(top, see >> i & 1 ? __uint_as_float(v[i]) : kNone);
    }
    return top;
}

// The reference that a row's first block sets.  Rounded up, so that no weight exceeds 2^kBaseMany.
__device__ __noinline__ float first_reference(float m, float c, Seen seen, uint32_t s_at) {
    const float top = largest(seen, s_at);
    return top > kNone ? __fsub_ru(__fmul_ru(top, c), kBaseMany) : m;
}

// The reference of this thread's row moved so that the block's weights, which add up to `sum`, will add up to 2^kUpSum or
// 2^kDownSum, l and the row of O rescaled, for the rows of a warp that need it (the others keep theirs): (reference, l).
// Out of line: it runs where logits change by many orders.
template <int D>
__device__ __noinline__ float2 moved(float m, float l, float sum, float c, Seen seen, uint32_t s_at, uint32_t o_at) {
    const bool need = misplaced(sum, l), past = need && sum == -kNone;
    float to = m;
    if (need) to = fmaxf(sub_rn(m, kDrop), __fadd_ru(m, log2f(sum) - (sum > 1.0f ? kUpSum : kDownSum)));
    if (__any_sync(kFullMask, past)) {                    // past fp32: by the largest
        const float top = largest(seen, s_at);
        if (past) to = fmaxf(m, __fsub_ru(__fmul_ru(top, c), kBaseMany));
    }
    const float less = exp2_approx(sub_rn(m, to));
#pragma unroll 1
    for (int q = 0; q < D / 32; ++q) {
        uint32_t v[32];
        __syncwarp();
        tmem_load32(o_at + 32 * q, v);
        tmem_wait_load(v);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(mul_rn(__uint_as_float(v[i]), less));
        tmem_store32(o_at + 32 * q, v);
    }
    tmem_wait_store();
    __syncwarp();
    return make_float2(to, mul_rn(l, less));
}

// The weights of a block some of whose keys a row does not see: their sum; with `store` they go over S.
__device__ __noinline__ float masked_weights(float m, float c, Seen seen, uint32_t s_at, bool store) {
    float sum = 0.0f;
#pragma unroll 1
    for (int q = 0; q < kKeys / 32; ++q) {
        uint32_t v[32], h[16];
        __syncwarp();
        tmem_load32(s_at + 32 * q, v);
        tmem_wait_load(v);
        const uint32_t see = seen.of(q);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float x = __fmaf_rn(__uint_as_float(v[i]), c, -m), y = exp2_approx(see >> i & 1 ? x : kNone);      // (no branch)
            sum = add_rn(sum, y);
            v[i] = __float_as_uint(y);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) h[i] = pack_f16(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
        __syncwarp();
        if (store) tmem_store16(s_at + 16 * q, h);
    }
    return sum;
}

template <int D>
__global__ void __launch_bounds__(kThreadsMany, 1) k_attend_many(const AttendArgs a) {
    using M = Many<D>;
    extern __shared__ __align__(1024) uint8_t smem[];     // (where it is not, the CTA gives up below)
    float* const factors = reinterpret_cast<float*>(smem + M::factor);
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + M::bars);
    uint32_t* const tmem_base = reinterpret_cast<uint32_t*>(bars + kBars);
    volatile int* const lost = reinterpret_cast<volatile int*>(tmem_base + 1);
    uint32_t* const there = tmem_base + 2;                // [4]: the tiles of a block that have a page

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2, t = threadIdx.x & 127;
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_base)),
                     "r"(M::cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < kBars; ++i) {
            const bool threads = (i >= kKFull && i < kKEmpty) || (i >= kVFull && i < kVEmpty) || (i >= kPFull && i < kOFull) || i >= kRaw;
            mbar_init(bars + i, i == kQFull ? 256 : threads ? 128 : i == kQEmpty ? 9 : 1);       // (the last S, and 8 softmax warps)
        }
        *lost = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    pdl_trigger();
    pdl_wait();
    constexpr uint32_t tmem = 0;                          // all of it: the products' operands are constants
    const int G = a.Hq / a.cache.Hkv, per_page = a.cache.page_size / 16;
    Spot* const spots = reinterpret_cast<Spot*>(smem + M::spots);
    Run& run = reinterpret_cast<Run*>(smem + M::runs)[warp];
    Cut* const cut = cuts<D, kRows>(a, gridDim.x) + blockIdx.x;
    if (warp < 3) {
        const Shares<Keys> shares(a);
        const int64_t ctas = runs_of(shares.total, gridDim.x), i = static_cast<int64_t>(blockIdx.x) - 1 + warp;
        const Spot p = spot_of(a, shares, i < 0 ? 0 : i < ctas ? quotient(shares.total * i, ctas) : shares.total);
        if (lane == 0) spots[warp] = p;
        if (warp == 1 && lane == 0) cut->last = p.blk > 0 ? static_cast<int>(quotient(p.until * ctas - 1, shares.total)) : 0;
    }
    __syncthreads();
    if (lane == 0) run.start(a, spots[1], spots[2]);
    if (threadIdx.x == 0) {                               // a group is cut at this run's start, and here first?
        const Spot& p = spots[1];
        const bool is = p.blk > 0 && !(spots[0].group_of(p) && spots[0].blk > 0);
        cut->n = is ? run.s.n : 0, cut->row0 = run.s.row0, cut->h = p.h, cut->rt = p.rt;
    }
    __syncwarp();
    auto step = [&]() {
        __syncwarp();
        if (lane == 0) run.step(a, spots[2]);
        __syncwarp();
    };
    uint32_t n = 0, items = 0;                            // blocks and parts with blocks so far
    bool ok = *tmem_base == 0 && smem_addr(smem) % 1024 == 0;

    if (wg >= 3) {
        // ---- producers: of keys and Q of tile A, of values and Q of tile B
        registers_down<kProducerRegisters>();
        // A thread takes 32 elements of a token: kPairs threads a token, kTokens tokens at once, kPairs turns a block.
        constexpr int kPairs = D / 32, kTokens = 128 / kPairs;
        const int token = t / kPairs, pair = t % kPairs, row = token % 16;
        // 32 elements are four 16-byte pieces of the swizzled row; the upper half's threads begin with the third, so that 8
        // threads' pieces lie in 8 bank groups
        const int upper = pair >> 1;
        const uint32_t piece = upper * M::half + token * 128 + (((pair & 1) * 4 ^ 2 * upper ^ token & 7) << 4);    // the j-th: ^ j << 4
        const int skip_pages = 8 / per_page, skip_tiles = 8 % per_page;
        const bool values = wg == 4;
        uint64_t *const full = bars + (values ? kVFull : kKFull), *const empty = bars + (values ? kVEmpty : kKEmpty);
        uint8_t* const ring = smem + (values ? M::v : M::k);
        const int codes = (values ? 9 * D : 0) + row * (D / 2) + pair * 16;       // in a tile
        const int scales = (values ? 17 * D : 8 * D) + row * (D / 16) + pair * 2;
        uint4 w[kPairs];                                  // the next block's codes and scales
        uint32_t sc[kPairs];
        uint32_t raws = 0;                                // copies of queries so far
        for (; ok && run.more; step()) {
            const Item it(a, run.s, run.at.rt);
            const int h = run.at.h, from = run.at.blk, to = run.to(it, spots[2]);
            if (from == to) continue;
            const int pos0 = it.s.len - it.s.n;
            const int seen_lo = a.window > 0 ? max(0, pos0 + it.first - a.window + 1) : 0;
            // a lane below 8 holds a tile of the block whose loads come next: its number (tl), its page's place in the table
            // and its place in the page, counted along
            const int tiles_end = min((it.s.len + 15) / 16, it.j0 / 16 + to * 8);
            int tl = it.j0 / 16 + from * 8 + (lane & 7);
            const int32_t* table = a.pages + run.at.b * a.width + tl / per_page;
            int tip = tl % per_page;
            auto page_of = [&]() { return tl < tiles_end ? __ldg(table) : -1; };
            // its number in the cache (-1: none); the next block's tile
            auto place_of = [&](int32_t page) {
                const int place = page >= 0 && page < a.cache.pages ? (page * a.cache.Hkv + h) * per_page + tip : -1;
                tl += 8, tip += skip_tiles, table += skip_pages;
                if (tip >= per_page) tip -= per_page, ++table;
                return place;
            };
            auto load = [&](int at) {
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    const int x = __shfl_sync(kFullMask, at, (i * kTokens + token) / 16);
                    const uint8_t* const tile = a.cache.data + static_cast<int64_t>(x) * kRecord<D>;
                    load_if(x >= 0, tile + codes, tile + scales, w[i], sc[i]);
                }
            };
            int at = place_of(page_of());
            load(at);
            // ---- this item's queries: copied as they are, a row a thread, then made f16 where they lie (its pieces in their
            // swizzled order), D / 8 threads a row
            if (items > 0) ok = wait(bars + kQEmpty, (items - 1) & 1, lost);
            const int tile = values ? 1 : 0;
            if (ok && tile * 128 < it.rows) {
                uint8_t* const dst = smem + M::q + tile * M::tile;
                int query, head;
                split_row(it.s.n, G, run.at.rt * kRows + min(tile * 128 + t, it.rows - 1), &query, &head);
                const uint16_t* const src = static_cast<const uint16_t*>(a.q) + (it.s.row0 + query) * a.q_stride +
                                            (static_cast<int64_t>(h) * G + head) * D;
                mbar_expect_tx(bars + kRaw + tile, 2 * D);
#pragma unroll
                for (int i = 0; i < D / 64; ++i) bulk_copy(dst + i * M::half + t * 128, src + 64 * i, 128, bars + kRaw + tile);
                float dec = 1.0f, enc;
                if (a.cache.k_mode != NVFP4_GAMAX_NONE)
                    global_scales(__ldg(a.cache.k_gamax + (a.cache.k_mode == NVFP4_GAMAX_ROW_GIVEN ? h : 0)), a.cache.bound, enc, dec);
                const float all = mul_rn(mul_rn(fabsf(a.scale), kLog2e), dec);
                ok = wait(bars + kRaw + tile, raws++ & 1, lost);
                constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
                const int q = lane % kLanes;
                if (ok) {
#pragma unroll 2
                    for (int i = 0; i < 32; i += kAtOnce) {
                        const int in_tile = (warp & 3) * 32 + i + lane / kLanes, r = tile * 128 + in_tile;
                        uint8_t* const at = dst + q / 8 * M::half + in_tile * 128;
                        const uint4 u = *reinterpret_cast<const uint4*>(at + (q & 7) * 16);
                        uint32_t top = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(0u, u.x), u.y), u.z), u.w);
                        top = max(top << 16, top & 0xFFFF0000u);
#pragma unroll
                        for (int o = kLanes / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(kFullMask, top, o));      // all have read
                        const int ex = min(max(static_cast<int>(top >> 23) - 127, -112), 126) - 14;
                        const float down = copysignf(power_of_two(-ex), a.scale);
                        if (q == 0) factors[r] = mul_rn(power_of_two(ex), all);
                        const uint32_t v[4] = {u.x, u.y, u.z, u.w};
                        uint32_t o[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)           // rows past the group's last are zeros
                            o[k] = r < it.rows ? pack_f16(mul_rn(__uint_as_float(v[k] << 16), down), mul_rn(__uint_as_float(v[k] & 0xFFFF0000u), down)) : 0u;
                        *reinterpret_cast<uint4*>(at + (((q & 7) ^ (in_tile & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
            }
            if (!ok) break;
            fence_async();
            arrive(bars + kQFull);
            // ---- its blocks
            for (int blk = from; blk < to; ++blk, ++n) {
                const int st = n & 1, j0 = it.j0 + blk * kKeys;
                const int32_t page = page_of();               // of the next block's tile
                if (values && (j0 < seen_lo || j0 + kKeys > it.s.len)) {      // some were perhaps never written
#pragma unroll
                    for (int i = 0; i < kPairs; ++i) {
                        const int j = j0 + i * kTokens + token;
                        if (j < seen_lo || j >= it.s.len) sc[i] = 0;
                    }
                }
                if (n >= 2 && !(ok = wait(empty + st, (n >> 1 & 1) ^ 1, lost))) break;
                uint8_t* const base = ring + st * M::tile;
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    const uint32_t u = e4m3_pair(sc[i]);
                    const uint32_t s0 = __byte_perm(u, u, upper ? 0x3232 : 0x1010), s1 = __byte_perm(u, u, upper ? 0x1010 : 0x3232);
                    const uint32_t x[4] = {upper ? w[i].z : w[i].x, upper ? w[i].w : w[i].y, upper ? w[i].x : w[i].z,
                                           upper ? w[i].y : w[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t o[4];
                        decode4(x[j], j < 2 ? s0 : s1, o);
                        *reinterpret_cast<uint4*>(base + (piece ^ j << 4) + i * kTokens * 128) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
                const unsigned have = __ballot_sync(kFullMask, lane < 8 && at >= 0);
                if (t == 0 && !values) there[n & 3] = have;
                fence_async();
                arrive(full + st);
                at = place_of(page);
                load(at);
            }
            ++items;
        }
    } else if (wg == 0) {
        // ---- products (the oldest warp: the first to issue)
        registers_down<kProductRegisters>();
        if (warp == 0) {
        const uint32_t el = elect_one();
        const uint32_t id_s = idesc_f16(128, kKeys, false), id_o = idesc_f16(128, D, true);
        const uint32_t base = smem_addr(smem) >> 4;
        // (tile and stage are constants where these are called)
        auto qk = [&](int tile, int st) {
            const uint32_t q = base + ((M::q + tile * M::tile) >> 4) + (1u << 16), k = base + ((M::k + st * M::tile) >> 4) + (1u << 16);
            unrolled<D / 16>([&](auto step) {
                constexpr int i = decltype(step)::value, at = (i / 4 * M::half + i % 4 * 32) >> 4;
                mma_ss<at, at>(el, tmem + M::s_col + tile * kKeys, q, k, id_s, i > 0);
            });
            commit_warp<1>(el, bars + kSFull + tile);
        };
        auto pv = [&](int tile, int st, bool first) {
            const uint32_t v = base + ((M::v + st * M::tile) >> 4) + (static_cast<uint32_t>(M::half >> 4) << 16);
            unrolled<kKeys / 16>([&](auto step) {
                constexpr int i = decltype(step)::value;
                mma_ts<(i * 2048 >> 4)>(el, tmem + M::o_col + tile * D, tmem + M::s_col + tile * kKeys + i * 8, v, id_o, i > 0 ? 1u : !first);
            });
        };
        uint32_t turn_b = 0;                              // blocks that tile B took part in
        for (; ok && run.more; step()) {
            const Item it(a, run.s, run.at.rt);
            const int from = run.at.blk, to = run.to(it, spots[2]);
            if (from == to) continue;
            const bool two = it.rows > 128;
            if (!(ok = wait(bars + kQFull, items & 1, lost))) break;
            if (!(ok = wait(bars + kKFull + (n & 1), n >> 1 & 1, lost))) break;
            fence_after();
            auto start = [&](auto stage) {
                constexpr int st = decltype(stage)::value;
                qk(0, st);
                if (two) qk(1, st);
                commit_warp<1>(el, bars + kKEmpty + st);
                if (from + 1 == to) commit_warp<1>(el, bars + kQEmpty);
            };
            if (n & 1) start(Constant<1>());
            else start(Constant<0>());
            // block blk's O, the next one's S
            auto turn = [&](auto stage, int blk) {
                constexpr int st = decltype(stage)::value, st1 = st ^ 1;
                const bool more = blk + 1 < to;
                if (!wait(bars + kVFull + st, n >> 1 & 1, lost)) return false;
                if (more && !wait(bars + kKFull + st1, (n + 1) >> 1 & 1, lost)) return false;
                if (!wait(bars + kPFull, n & 1, lost)) return false;
                fence_after();
                pv(0, st, blk == from);
                if (more) {
                    qk(0, st1);
                } else {
                    commit_warp<1>(el, bars + kOFull);
                }
                if (two) {
                    if (!wait(bars + kPFull + 1, turn_b++ & 1, lost)) return false;
                    fence_after();
                    pv(1, st, blk == from);
                    if (!more) commit_warp<1>(el, bars + kOFull + 1);
                }
                commit_warp<1>(el, bars + kVEmpty + st);
                if (more) {
                    if (two) qk(1, st1);
                    commit_warp<1>(el, bars + kKEmpty + st1);
                    if (blk + 2 == to) commit_warp<1>(el, bars + kQEmpty);      // the next item's queries may come
                }
                ++n;
                return true;
            };
            for (int blk = from; ok && blk < to; ++blk) ok = n & 1 ? turn(Constant<1>(), blk) : turn(Constant<0>(), blk);
            if (!ok) break;
            ++items;
        }
        }
    } else {
        // ---- softmax of a tile: this thread's row
        registers_up<kSoftmaxRegisters>();
        const int tile = wg - 1;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;           // 32 lanes of tensor memory a warp
        const uint32_t s_at = tmem + lanes + M::s_col + tile * kKeys, o_at = tmem + lanes + M::o_col + tile * D;
        uint32_t turn = 0, mine = 0;                      // blocks and items that this tile took part in
        for (; ok && run.more; step()) {
            const Item it(a, run.s, run.at.rt);
            const int h = run.at.h, from = run.at.blk, to = run.to(it, spots[2]);
            const int r = tile * 128 + t;
            int query, head;
            split_row(it.s.n, G, min(run.at.rt * kRows + r, it.s.n * G - 1), &query, &head);
            float m = kLowest, l = 0.0f;
            float c = 0.0f;
            if (from < to) {                              // (a tile that has no rows waits too: it must not fall a part behind)
                if (!(ok = wait(bars + kQFull, items & 1, lost))) break;
                c = factors[r];
                __syncwarp();
                if (lane == 0) arrive(bars + kQEmpty);
            }
            if (from < to && tile * 128 < it.rows) {
                const int p = it.s.len - it.s.n + query;
                const int hi = a.causal ? min(it.s.len, max(p + 1, 0)) : it.s.len, lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
                for (int blk = from; blk < to; ++blk, ++turn) {
                    const uint32_t block = n + blk - from;
                    const int j0 = it.j0 + blk * kKeys;
                    // (a tile that sat out an item keeps its own count of S and P)
                    if (!(ok = wait(bars + kSFull + tile, turn & 1, lost))) break;
                    fence_after();
                    const uint32_t have = there[block & 3];
                    const bool whole = __all_sync(kFullMask, have == 0xFFu && j0 >= lo && j0 + kKeys <= hi);
                    const Seen seen{lo - j0, hi - j0, have};
                    const bool fresh = blk == from;       // the reference is this block's
                    if (fresh) m = first_reference(m, c, seen, s_at);
                    if (whole) {
                        uint32_t p16[kKeys / 2];
                        for (int again = 0;; ++again) {
                            uint64_t sum = 0;                     // two fp32
                            uint32_t v[2][32];
                            tmem_load32(s_at, v[0]);
#pragma unroll
                            for (int q = 0; q < kKeys / 32; ++q) {
                                tmem_wait_load(v[q & 1]);
                                if (q + 1 < kKeys / 32) tmem_load32(s_at + 32 * (q + 1), v[(q + 1) & 1]);
#pragma unroll
                                for (int i = 0; i < 32; i += 2) {
                                    float y0, y1;
                                    unpack2(fma2(pack2(__uint_as_float(v[q & 1][i]), __uint_as_float(v[q & 1][i + 1])), pack2(c, c),
                                                 pack2(-m, -m)), y0, y1);
                                    y0 = exp2_approx(y0), y1 = exp2_approx(y1);
                                    sum = add2(sum, pack2(y0, y1));
                                    p16[16 * q + i / 2] = pack_f16(y0, y1);
                                }
                            }
                            float a0, a1;
                            unpack2(sum, a0, a1);
                            const float more = add_rn(a0, a1);
                            if (again || !__any_sync(kFullMask, misplaced(more, l))) {
                                l = add_rn(l, more);
                                break;
                            }
                            const float2 x = moved<D>(m, l, more, c, seen, s_at, o_at);
                            m = x.x, l = x.y;
                        }
                        tmem_store32(s_at, p16);
                        tmem_store32(s_at + 32, p16 + 32);
                    } else {
                        float some = fresh ? 1.0f : masked_weights(m, c, seen, s_at, false);
                        if (some == 0.0f) some = 1.0f;        // a row that sees nothing here: its reference stays
                        if (__any_sync(kFullMask, misplaced(some, l))) {
                            const float2 x = moved<D>(m, l, some, c, seen, s_at, o_at);
                            m = x.x, l = x.y;
                        }
                        l = add_rn(l, masked_weights(m, c, seen, s_at, true));
                    }
                    tmem_wait_store();
                    fence_before();
                    arrive(bars + kPFull + tile);
                }
                if (!ok) break;
                if (!(ok = wait(bars + kOFull + tile, mine & 1, lost))) break;
                fence_after();
                ++mine;
            }
            if (from < to) n += to - from, ++items;
            // ---- the row's output (a group without keys gives zeros), or its part of it
            if (tile * 128 < it.rows) {
                const bool complete = from == 0 && to == it.blocks;
                float* const part = reinterpret_cast<float*>(a.workspace) +
                                    (static_cast<int64_t>(blockIdx.x) * 2 + (from > 0 ? 0 : 1)) * kPart<D, kRows>;
                const Finish f(a, h * G + head, h, m, l);
                const bool wide = !complete || a.out_dtype == NVFP4_F32;
                const int64_t row = (it.s.row0 + query) * a.Hq + h * G + head;
                const uint64_t base = r >= it.rows ? 0
                                      : complete   ? reinterpret_cast<uint64_t>(a.out) + row * D * (wide ? 4 : 2)
                                                   : reinterpret_cast<uint64_t>(part + r * D);
                const float by = complete ? f.by : 1.0f;
                if (complete && a.lse && r < it.rows) a.lse[row] = f.lse;
                // 128 bytes of each of the warp's rows at a time, through shared memory, so that 8 lanes write a row's (a row
                // a lane kept the stores of 256 rows busy for 3 to 5 us)
                uint8_t* const out = smem + M::stage + (warp - 4) * 32 * 128;
                uint8_t* const mine = out + lane * 128;
#pragma unroll 1
                for (int q = 0; q < (wide ? D / 32 : D / 64); ++q) {
                    __syncwarp();                         // the rows before are read
#pragma unroll 1
                    for (int half = 0; half < (wide ? 1 : 2); ++half) {
                        uint32_t v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0u;
                        if (from < to) {
                            __syncwarp();
                            tmem_load32(o_at + 32 * (wide ? q : 2 * q + half), v);
                            tmem_wait_load(v);
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(mul_rn(__uint_as_float(v[i]), by));
                        if (wide) {
#pragma unroll
                            for (int p = 0; p < 8; ++p)
                                *reinterpret_cast<uint4*>(mine + ((p ^ (lane & 7)) << 4)) = make_uint4(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
                        } else {
#pragma unroll
                            for (int p = 0; p < 4; ++p) {
                                uint32_t w[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(v[8 * p + 2 * i]), __uint_as_float(v[8 * p + 2 * i + 1]));
                                    w[i] = *reinterpret_cast<const uint32_t*>(&x);
                                }
                                *reinterpret_cast<uint4*>(mine + ((p + 4 * half ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int x = 4 * i + (lane >> 3);
                        const uint64_t to_row = __shfl_sync(kFullMask, base, x);
                        const uint4 u = *reinterpret_cast<const uint4*>(out + x * 128 + (((lane & 7) ^ (x & 7)) << 4));
                        if (to_row) *reinterpret_cast<uint4*>(to_row + q * 128 + (lane & 7) * 16) = u;
                    }
                }
                if (!complete && r < it.rows) *reinterpret_cast<float2*>(part + kRows * D + 2 * r) = make_float2(m, l);
                __syncwarp();
                fence_before();
            }
        }
        if (!ok) {                                        // NaN to the rows of this run, and to its parts' denominators
            __syncwarp();
            if (lane == 0) run.start(a, spots[1], spots[2]);
            __syncwarp();
            for (; run.more; step()) {
                const Item it(a, run.s, run.at.rt);
                const int h = run.at.h, from = run.at.blk, r = tile * 128 + t;
                if (r >= it.rows) continue;
                int query, head;
                split_row(it.s.n, G, run.at.rt * kRows + r, &query, &head);
                if (from == 0 && run.to(it, spots[2]) == it.blocks) {
                    const float nan = __int_as_float(0x7FC00000);
                    const Finish f(a, h * G + head, h, 0.0f, nan);
                    for (int d = 0; d < D; d += 4) {
                        float y[4] = {nan, nan, nan, nan};
                        f.store(a, it.s.row0 + query, h * G + head, d, y);
                    }
                } else {
                    float* const part = reinterpret_cast<float*>(a.workspace) +
                                        (static_cast<int64_t>(blockIdx.x) * 2 + (from > 0 ? 0 : 1)) * kPart<D, kRows>;
                    *reinterpret_cast<float2*>(part + kRows * D + 2 * r) = make_float2(0.0f, __int_as_float(0x7FC00000));
                }
            }
        }
    }
    if (!ok) settle();
    fence_before();
    __syncthreads();
    if (warp == 0) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(M::cols));
    }
}

template <int D>
cudaError_t launch_many(const AttendArgs& a, cudaStream_t s) {
    static thread_local int dev_of = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev_of != dev) {
        const cudaError_t e = cudaFuncSetAttribute(k_attend_many<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Many<D>::bytes);
        if (e != cudaSuccess) return e;
        dev_of = dev;
    }
    const int grid = sm_count();
    cudaError_t e = launch_pdl(k_attend_many<D>, dim3(static_cast<unsigned>(grid)), dim3(kThreadsMany), Many<D>::bytes, s, a);
    if (e == cudaSuccess) e = launch_join<D, kRows>(a, grid, s);
    return e;
}

}  // namespace

int64_t attend_many_workspace(const AttendArgs& a) {
    return static_cast<int64_t>(sm_count()) * (2 * kRows * (a.cache.D + 2) * 4 + static_cast<int64_t>(sizeof(Cut)));
}

cudaError_t launch_attend_many(const AttendArgs& a, cudaStream_t s) {
    return a.cache.D == 64 ? launch_many<64>(a, s) : launch_many<128>(a, s);
}

}  // namespace nvfp4
