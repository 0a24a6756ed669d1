// window.cu -- attention of a ragged batch of tokens to a sliding window and to the
// first tokens ("sinks") over the paged FP8 cache: single tokens to prompt chunks.
//
// The token at position p sees the keys j <= p with p - j < window or j < sinks. The
// query rows that share a kv head are the sequence's tokens x the group of query heads;
// they are taken in items of at most 256, and an item walks the blocks that any of its
// rows sees: those of the sinks, then those from the first row's window to the last
// row's position. No block between the two is read.
//
//   S = Q_fp8 K_fp8^T                 tcgen05 kind::f8f6f4, 128 rows x 128 keys
//   x = S k_scale q_scale scale log2e, -inf where the row does not see the key
//   P = 2^(x - m + 7), L += sum P     one thread per row, FP32
//   O += FP16(P) V                    tcgen05 kind::f16, P from tensor memory
//   out = BF16(O v_scale / L)
//
// The numbers are tree.cu's: P in FP16 (half a step 2^-11), V's codes as FP16 exactly. m
// is raised only where P would leave FP16: the sum of a thread's 32 P, which it forms
// anyhow, tells (2^15 at most); no maximum is looked up but then and at an item's begin.
//
// Two softmax warpgroups, each with an S and an O of its own in tensor memory (2 x 128
// + 2 x 128 columns); P lies over its S's columns. A step is one tile of 128 rows and a
// block of 128 keys, and the steps alternate between the warpgroups: an item of more than
// 128 rows is two tiles, one a warpgroup, and every block makes two steps; in a smaller
// one both warpgroups work on the same rows and take the blocks in turn, and their O, m
// and l are joined at its end. So S of a warpgroup's next step is computed while the
// other works, K, V and V's conversion serve 256 rows of a prompt, and the warpgroups
// share nothing inside an item.
//   warps 0-7        softmax (thread = row = tensor memory lane)
//   warp 8           K and V blocks by TMA, key scales by cp.async
//   warp 9           issues S and P V
//   warp 10          Q rows and scales of the next item
//   warp 11          the run's items, one after another, for all others; zeros where a token sees nothing
//   warps 12-15      V codes to FP16 in shared memory, zeros where no row sees the key
// The issuing warp issues S of step j + 2 behind P V of step j, so that the tensor core
// itself keeps them apart where they share columns, and an S that is complete says that
// the warpgroup's last P V is. (What PTX names as kept in order are MMAs of one accumulator
// and shape, which these are not: it rests on an SM's tensor core taking one thread's MMAs
// one after another in the order of their issue. Were it not so, S would have to wait
// for P V's commit, and tests that compare repeated calls bit for bit would differ.)
//
// An item of at most 64 rows (a decoding request's: one token x the group) stands in the
// tile twice, and either copy's warps take a half of the block's keys: with one copy most of
// a warpgroup's warps would have no rows (64 decoding requests then 127 us, with two 116, with
// four copies of 32 rows 117). The copies have an O, an m and an l of their own and are joined
// with the warpgroups' at the end.
//
// Loops are rolled (32 scores at a time) and what is rare lies behind branches that are
// marked so: the parts run at once out of one instruction cache.
//
// What bounds it, on 152 SMs: prompts, the chain of a step's hand-overs and the softmax
// warps' part of it. A step of 128 x 128 takes a warpgroup 2500 clocks for its P (1700 with
// nothing else on the SM; 1140 if the other warpgroup rests, too), 700 of waiting for P V
// and the next S and 400 around them, so that with two in flight the tensor core has work
// 42% of the time. Without the exponentials it would be 3% faster, without V's conversion
// 5%, without the key scales 6%. Two prompts of 5000 tokens, 8 x 12 heads, window 4096: 612
// us (1.27 PFLOP/s). Six chunks of up to 509 tokens beside 31 decoding requests, window
// 1000: 154 us; of an item's 32000 clocks 10000 go to its begin, its last P V and its output.
// Decoding, the blocks' reads: 64 requests of 8 x 12 heads, window 4096, 550 MB in 115 us
// (111 in a graph, 5.0 TB/s), four requests of 110000 tokens 170 us (5.5 TB/s); an item ends
// with 10000 clocks in which only the next three blocks are read. One token of one request:
// 14.3 us, 11.5 in a graph, launches, schedule and one pass through every part.
//
// The items in (sequence, kv head, row) order are dealt to the CTAs in runs of equal
// weight: a step counts 1, an item kItemCost besides. Items that a run's end cuts leave
// FP32 partial sums, which a second kernel joins.
#include "attend.cuh"

#include <algorithm>
#include <cmath>
#include <cstddef>

namespace pa {
namespace {

constexpr int kD = 128;
constexpr int kBS = 128;
constexpr int kMaxGroup = 128;
constexpr int kMaxB = 1024;
constexpr int kMaxCtas = 192;
constexpr int kTileRows = 128;
constexpr int kItemRows = 2 * kTileRows;
constexpr int kTile = kBS * kD;              // bytes of a block of codes
// What g_mul stands for: the product, 2^22 (1 + kItemRows / G) + G + kItemRows at most, in 32 bits
// for every G (1 is the worst), and its excess of n / 2^22 below 1 / G.
static_assert((1ull << 22) * (1 + kItemRows) + kMaxGroup + kItemRows < (1ull << 32), "n g_mul leaves 32 bits");
static_assert(kMaxGroup * (kMaxGroup + kItemRows) < (1 << 22), "n g_mul >> 22 passes n / G");
// K blocks, V blocks as codes and as FP16. The key scales' ring needs no barrier that
// says a slot is free: block i + 8 is requested once K block i + 5 is free, i.e. its S
// complete; that was issued behind block i + 3's P V, so that block i's softmax is done.
constexpr int kKStages = 3, kVStages = 2, kHStages = 2, kSStages = 8;
constexpr int kProdWarp = 8, kMmaWarp = 9, kQWarp = 10, kSegWarp = 11, kConvWarp = 12, kConvWarps = 4;
constexpr int kThreads = (kConvWarp + kConvWarps) * 32;
constexpr int kChunk = 32;                   // scores a softmax thread holds at once
constexpr uint32_t kTmemCols = 512, kSCol = 2 * kD;   // O of either warpgroup, then S (and P)
constexpr float kShift = 7.0f;               // log2 units
constexpr float kRaise = 3.0f;
constexpr float kLimit = 0x1p15f;            // of a chunk's sum; one that passes it has a P of 2^(3 + 7)
constexpr int kItemCost = 5;                 // of an item besides its steps, in steps (3 to 11 tried)
// The shortest run (2 at least: describe_cut). One token, 8 x 12 heads, window 1024: 16.5 us,
// with 6 18.5, with 12 22.4.
constexpr int kMinRun = 2;
constexpr int kSegs = 4;                     // items ahead of the slowest part
// Entries of the schedule in shared memory: an item each while the batch's number no
// more than 512 a kv head, else 2, 4, .. one behind another.
constexpr int kMaxEntries = kMaxB + 512;

// What the joining kernel has to know of the item at the begin of a run.
struct Cut {
    int h, row0, rows, tok0;                 // rows 0: nothing to join
    int c0, c1;                              // the runs that have its first and its last block
    int slot0, b;                            // where run c0's part lies
};

// Workspace: error word, a Cut per CTA, then per CTA two partial items: O [rows][128],
// m and l [rows]. Slot 2 c is of run c's first item, slot 2 c + 1 of its last.
constexpr size_t kCutOff = 256;
constexpr size_t kPartOff = kCutOff + kMaxCtas * sizeof(Cut);

struct WindowParams {
    const uint8_t* q;
    const float* q_scale;
    const float* k_scale;
    const float* v_scale;
    const int *bt, *act, *cu;
    __nv_bfloat16* out;
    int* err;
    Cut* cuts;
    float* part;
    int part_rows;                           // rows of a partial item
    int B, T, max_tokens, NQ, NKV, G;
    uint32_t g_mul;                          // 2^22 / G + 1: n / G = n g_mul >> 22 for n < G + kItemRows
    uint64_t g_inv;                          // 2^64 / G + 1 (G > 1)
    int one_item;                            // a sequence makes one item at most (no scan: 0.7 us of 15)
    int64_t num_blocks;
    int max_blocks, layout, ctas;
    int window, sinks;
    float scale_log2;
};

struct Item {
    int row0, rows;
    int first, last;                         // positions of its first and last row's token
    int lo, sink_blocks, blocks;             // first block of the windows, blocks of the sinks before it, in all
};

struct Seg {
    Item x;
    int b, h;
    int t0, t1;                              // its blocks that this run has
    int tok;                                 // the row of the sequence's first token
    int first_of_run;
};

struct WindowSmem {
    alignas(1024) uint8_t k[kKStages][kTile];
    alignas(1024) uint8_t v[kVStages][kTile];
    alignas(1024) uint8_t vh[kHStages][2][kTile];   // FP16, channels 0-63 and 64-127
    alignas(1024) uint8_t q[2 * kTile];             // of either tile
    alignas(16) float ks[kSStages][kBS];
    alignas(16) float qs[2][kItemRows];             // by item parity, as vs
    alignas(16) float vs[2][kD];
    float m[2 * kTileRows], l[2 * kTileRows];       // of the warpgroups' threads
    float4 join[kTileRows * 8];              // 32 or 64 channels of the lanes' rows
    float inv[kTileRows];                    // 1 / L of an item's rows
    // per sequence: position and row of its first token that sees a key, query rows a
    // kv head; entries before it
    int pos[kMaxB], tok[kMaxB], rows[kMaxB], first[kMaxB + 1];
    uint32_t cum[kMaxEntries + 1];           // weights before each entry, of one kv head
    uint64_t k_full[kSStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
    uint64_t h_full[kHStages], h_empty[kHStages];
    uint64_t s_full[2], p_full[2], o_full[2], q_full, q_empty, joined, drain, seg_full[kSegs], seg_empty[kSegs];
    Seg segs[kSegs];                         // the run's items; t1 = 0: the end
    uint32_t scan[kThreads / 32];
    uint32_t tmem;
    int abort;
};
constexpr size_t kSmemBytes = offsetof(WindowSmem, abort) + sizeof(int) + 1024;   // (aligned by hand)
static_assert(kSmemBytes <= 232448, "window attention shared memory too large");

// ---- waits -----------------------------------------------------------------------
// wait_for with all but the first try marked as rare.
__device__ __forceinline__ bool await(uint64_t* bar, uint32_t parity, int* err, int code, volatile int* abort)
{
    return __builtin_expect(mbar_try_wait(bar, parity), 1) || wait_for(bar, parity, err, code, abort);
}

// ---- the schedule -----------------------------------------------------------------
// n / G
__device__ __forceinline__ int tokens_of(const WindowParams& p, int n)
{
    return p.G == 1 ? n : static_cast<int>(__umul64hi(static_cast<uint64_t>(n), p.g_inv));
}

__device__ __forceinline__ Item item_of(const WindowParams& p, int pos, int rows, int i)
{
    Item x;
    x.row0 = i * kItemRows;
    x.rows = min(rows - x.row0, kItemRows);
    x.first = pos + tokens_of(p, x.row0);
    x.last = pos + tokens_of(p, x.row0 + x.rows - 1);
    x.lo = max(x.first - p.window + 1, 0) / kBS;
    x.sink_blocks = min((p.sinks + kBS - 1) / kBS, x.lo);
    x.blocks = x.sink_blocks + x.last / kBS - x.lo + 1;
    return x;
}
// copies of an item's rows in the tile
__device__ __forceinline__ int copies_of(int rows) { return rows <= kTileRows / 2 ? 2 : 1; }
__device__ __forceinline__ int steps_a_block(int rows) { return rows > kTileRows ? 2 : 1; }
__device__ __forceinline__ uint32_t weight_of(const Item& x) { return x.blocks * steps_a_block(x.rows) + kItemCost; }
__device__ __forceinline__ int items_of(int rows) { return (rows + kItemRows - 1) / kItemRows; }

struct Run {
    uint32_t pos, hi;                        // of the weights of all heads
    uint32_t base;                           // where item (b, h, i) begins
    int b, h, i;
    bool fresh;
};

__device__ __forceinline__ int block_at(const Item& x, int t)
{
    return t < x.sink_blocks ? t : x.lo + t - x.sink_blocks;
}

// Chunks [a, b) of an item's block t that any of its rows sees: the others take no part.
// (In the two blocks at a window's ends half of the keys on average, of a few sinks one
// chunk: a window of 1000 of 10 blocks.)
struct Span {
    int a, b;
};
__device__ __forceinline__ Span chunks_of(const WindowParams& p, const Item& x, int t)
{
    const int k0 = block_at(x, t) * kBS, sink = p.sinks - k0;
    const int begin = sink > 0 ? 0 : max(x.first - p.window + 1 - k0, 0);
    const int end = t < x.sink_blocks ? sink : x.last + 1 - k0;
    return {begin / kChunk, min((end + kChunk - 1) / kChunk, kBS / kChunk)};
}

// blocks of an item before position `off` behind its first one
__device__ __forceinline__ int blocks_before(const Item& x, uint32_t off)
{
    return min(off > kItemCost ? static_cast<int>(off - kItemCost) / steps_a_block(x.rows) : 0, x.blocks);
}

// The run's next item with blocks [t0, t1) in it.
__device__ __forceinline__ bool next_seg(const WindowSmem& sm, const WindowParams& p, Run& r, Seg& s)
{
    while (r.pos < r.hi) {
        while (r.i >= items_of(sm.rows[r.b])) {
            r.i = 0;
            if (sm.rows[r.b] == 0 || ++r.h == p.NKV) {
                r.h = 0;
                ++r.b;
            }
        }
        s.x = item_of(p, sm.pos[r.b], sm.rows[r.b], r.i);
        s.b = r.b;
        s.h = r.h;
        s.tok = sm.tok[r.b];
        const uint32_t end = r.base + weight_of(s.x);
        s.t0 = blocks_before(s.x, r.pos - r.base);
        s.t1 = r.hi >= end ? s.x.blocks : blocks_before(s.x, r.hi - r.base);
        s.first_of_run = r.fresh;
        r.fresh = false;
        r.pos = min(end, r.hi);
        r.base = end;
        ++r.i;
        if (s.t0 < s.t1) return true;
    }
    return false;
}

// The run that starts at `pos` (below the total).
__device__ __forceinline__ Run locate(const WindowSmem& sm, const WindowParams& p, int group, uint32_t pos, uint32_t hi)
{
    Run r;
    r.pos = pos;
    r.hi = hi;
    r.fresh = true;
    int lo = 0, up = p.B - 1;                // the last sequence that starts at or before pos
    while (lo < up) {
        const int mid = (lo + up + 1) >> 1;
        if (p.NKV * sm.cum[sm.first[mid]] <= pos) lo = mid;
        else up = mid - 1;
    }
    r.b = lo;
    const int e0 = sm.first[lo], e1 = sm.first[lo + 1];
    const uint32_t start = sm.cum[e0], head = sm.cum[e1] - start;
    uint32_t rem = pos - p.NKV * start;
    r.h = static_cast<int>(rem / head);
    rem -= r.h * head;
    lo = e0;
    up = e1 - 1;                             // its last entry that starts at or before the rest
    while (lo < up) {
        const int mid = (lo + up + 1) >> 1;
        if (sm.cum[mid] - start <= rem) lo = mid;
        else up = mid - 1;
    }
    r.base = p.NKV * start + r.h * head + (sm.cum[lo] - start);
    r.i = (lo - e0) * group;
    for (;;) {
        const uint32_t w = weight_of(item_of(p, sm.pos[r.b], sm.rows[r.b], r.i));
        if (r.base + w > pos) return r;
        r.base += w;
        ++r.i;
    }
}

// Sum over the threads before this one, and over all; a barrier before and after.
__device__ __forceinline__ uint32_t block_scan(WindowSmem& sm, uint32_t mine, uint32_t& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sm.scan[warp] = x;
    __syncthreads();
    x -= mine;
    total = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
        const uint32_t s = sm.scan[i];
        if (i < warp) x += s;
        total += s;
    }
    return x;
}

// A sequence's rows in the batch and their positions. Its tokens are rows [tok, tok + n),
// at positions pos + i; those at negative positions and those behind max_tokens see
// nothing.
struct Sequence {
    int tok, n, skip, live;
    int pos;                                 // of token `skip`
};
__device__ __forceinline__ Sequence sequence(const WindowParams& p, int b)
{
    Sequence s;
    const int act = min(max(__ldg(p.act + b), 0), p.max_blocks * kBS);
    s.tok = min(max(__ldg(p.cu + b), 0), p.T);
    s.n = min(max(__ldg(p.cu + b + 1), s.tok), p.T) - s.tok;
    s.skip = max(s.n - act, 0);
    s.live = max(min(s.n, p.max_tokens) - s.skip, 0);
    s.pos = max(act - s.n, 0);
    return s;
}

// Fills the schedule's arrays; the weight of all kv heads, and the items an entry. 0 where
// cu_tokens decreases somewhere: rows would be counted twice, and the sums pass 32 bits.
__device__ uint32_t build_schedule(WindowSmem& sm, const WindowParams& p, int tid, int& group)
{
    constexpr int kSeqs = (kMaxB + kThreads - 1) / kThreads;
    int items = 0;
    bool decreases = false;
#pragma unroll
    for (int j = 0; j < kSeqs; ++j) {
        const int b = tid * kSeqs + j;
        if (b >= p.B) break;
        decreases = decreases || __ldg(p.cu + b + 1) < __ldg(p.cu + b);
        const Sequence s = sequence(p, b);
        sm.pos[b] = s.pos;
        sm.tok[b] = s.tok + s.skip;
        sm.rows[b] = s.live * p.G;
        items += items_of(s.live * p.G);
    }
    uint32_t total, entries;
    group = 1;
    if (p.one_item) {
        // a sequence an entry (of no weight if it has no rows)
        entries = p.B;
        for (int b = tid; b <= p.B; b += kThreads) sm.first[b] = b;
    } else {
        block_scan(sm, items, total);
        while (total > static_cast<uint32_t>(group) * (kMaxEntries - kMaxB)) group *= 2;
        uint32_t mine = 0;
#pragma unroll
        for (int j = 0; j < kSeqs; ++j) {
            const int b = tid * kSeqs + j;
            if (b < p.B) mine += (items_of(sm.rows[b]) + group - 1) / group;
        }
        uint32_t at = block_scan(sm, mine, entries);
#pragma unroll
        for (int j = 0; j < kSeqs; ++j) {
            const int b = tid * kSeqs + j;
            if (b >= p.B) break;
            sm.first[b] = at;
            at += (items_of(sm.rows[b]) + group - 1) / group;
        }
        if (tid == 0) sm.first[p.B] = entries;
    }
    if (__syncthreads_or(decreases)) {
        if (tid == 0) atomicOr(p.err, 16384);
        return 0;
    }
    uint32_t mine = 0;
    // thread i takes entries per i, per i + 1, .. and sums up its own
    const int per = (static_cast<int>(entries) + kThreads - 1) / kThreads;
    const int e0 = min(tid * per, static_cast<int>(entries)), e1 = min(e0 + per, static_cast<int>(entries));
    if (e0 < e1) {
        int lo = 0, up = p.B - 1;            // the last sequence with first <= e0
        while (lo < up) {
            const int mid = (lo + up + 1) >> 1;
            if (sm.first[mid] <= e0) lo = mid;
            else up = mid - 1;
        }
        for (int e = e0, b = lo; e < e1; ++e) {
            while (sm.first[b + 1] <= e) ++b;
            const int i0 = (e - sm.first[b]) * group, n = items_of(sm.rows[b]);
            sm.cum[e] = mine;
            for (int i = i0; i < min(i0 + group, n); ++i) mine += weight_of(item_of(p, sm.pos[b], sm.rows[b], i));
        }
    }
    const uint32_t before = block_scan(sm, mine, total);
    for (int e = e0; e < e1; ++e) sm.cum[e] += before;
    if (tid == 0) sm.cum[entries] = total;
    return total * p.NKV;
}

// Row r of an item in q and out: a row of tokens x heads.
__device__ __forceinline__ int64_t q_row(const WindowParams& p, int tok0, int h, int row)
{
    const int t = tokens_of(p, row);
    return static_cast<int64_t>(tok0 + t) * p.NQ + h * p.G + (row - t * p.G);
}

__device__ __forceinline__ float* part_of(const WindowParams& p, int cta, bool first)
{
    return p.part + (static_cast<int64_t>(cta) * 2 + (first ? 0 : 1)) * p.part_rows * (kD + 2);
}

// ---- the warps' parts ------------------------------------------------------------------
// The items of the run, from one warp to all others, each of which goes through them
// with a reader of its own.
__device__ void scheduler(WindowSmem& sm, const WindowParams& p, Run run, int lane)
{
    bool more = true;
    for (int i = 0; more; ++i) {
        Seg s;
        more = next_seg(sm, p, run, s);
        await(&sm.seg_empty[i % kSegs], ((i / kSegs) & 1) ^ 1, p.err, 2048, &sm.abort);
        if (!more) s.t1 = 0;
        if (lane == 0) {
            sm.segs[i % kSegs] = s;
            mbar_arrive(&sm.seg_full[i % kSegs]);
        }
        __syncwarp();
    }
}
constexpr int kSegReaders = 8 + 3 + kConvWarps;      // warps

// (A lane reads a word and all have it from there: what the warp does stays one even where
// a wait gave up and the entry is overwritten meanwhile.)
struct SegReader {
    int i = 0;
    __device__ __forceinline__ bool next(WindowSmem& sm, const WindowParams& p, Seg& s, int lane)
    {
        constexpr int kWords = sizeof(Seg) / 4;
        static_assert(kWords <= 32, "a word a lane");
        await(&sm.seg_full[i % kSegs], (i / kSegs) & 1, p.err, 4096, &sm.abort);
        const int mine = reinterpret_cast<const volatile int*>(&sm.segs[i % kSegs])[lane < kWords ? lane : 0];
        int* const words = reinterpret_cast<int*>(&s);
#pragma unroll
        for (int k = 0; k < kWords; ++k) words[k] = __shfl_sync(0xffffffffu, mine, k);
        if (lane == 0) mbar_arrive(&sm.seg_empty[i % kSegs]);
        ++i;
        return s.t1 > 0;
    }
};

__device__ void producer(WindowSmem& sm, const WindowParams& p, const CUtensorMap* tk, const CUtensorMap* tv, int lane)
{
    // Evicted first, also where a prompt's next items read the blocks again: two prompts of 5000
    // tokens so read 589 MB from memory for 91, but take 614 us for 627 (with the blocks evicted
    // like all else or as they were); 64 decoding requests 115 for 122.
    const uint64_t pol = l2_evict_first_policy();
    Seg s;
    int kc = 0, vc = 0;                      // blocks requested so far
    bool stop = false;
    SegReader segs;
    while (!stop && segs.next(sm, p, s, lane)) {
        const int* row = p.bt + static_cast<int64_t>(s.b) * p.max_blocks;
        int ids = 0;
        for (int t = s.t0; t < s.t1; ++t) {
            const int at = (t - s.t0) & 31;
            if (at == 0) {
                ids = t + lane < s.t1 ? __ldg(row + block_at(s.x, t + lane)) : 0;
                if (ids < 0 || ids >= p.num_blocks) ids = 0;
            }
            const int64_t blk = __shfl_sync(0xffffffffu, ids, at);
            const int x = p.layout == PA_LAYOUT_BSND ? s.h * kD : 0;
            const int y = static_cast<int>(p.layout == PA_LAYOUT_BSND ? blk * kBS : (blk * p.NKV + s.h) * kBS);
            const int kslot = kc % kKStages, vslot = vc % kVStages, sslot = kc % kSStages;
            if (!await(&sm.k_empty[kslot], ((kc / kKStages) & 1) ^ 1, p.err, 1, &sm.abort)) stop = true;
            if (__any_sync(0xffffffffu, stop)) {
                stop = true;
                break;
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(&sm.k_full[sslot], kTile);
                tma_load_2d(sm.k[kslot], tk, x, y, &sm.k_full[sslot], pol);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = lane + 32 * i;
                cp_async4(&sm.ks[sslot][j], p.k_scale + cache_row(p.layout, blk, j, s.h, kBS, p.NKV), 4);
            }
            cp_async_arrive_noinc(&sm.k_full[sslot]);
            ++kc;
            if (!await(&sm.v_empty[vslot], ((vc / kVStages) & 1) ^ 1, p.err, 2, &sm.abort)) stop = true;
            if (__any_sync(0xffffffffu, stop)) {
                stop = true;
                break;
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(&sm.v_full[vslot], kTile);
                tma_load_2d(sm.v[vslot], tv, x, y, &sm.v_full[vslot], pol);
            }
            ++vc;
            __syncwarp();
        }
    }
    // every copy has landed before this CTA's shared memory is given up
    for (int i = max(0, kc - kSStages); i < kc; ++i)
        mbar_wait_drain(&sm.k_full[i % kSStages], (i / kSStages) & 1, p.err, 256);
    for (int i = max(0, vc - kVStages); i < vc; ++i)
        mbar_wait_drain(&sm.v_full[i % kVStages], (i / kVStages) & 1, p.err, 256);
}

// V codes [key][channel] (128-byte swizzled rows) to FP16 in two chunks of 64 channels,
// swizzled the same way; keys that no row of the item sees become zeros, so that no
// stale code (a NaN among them) meets their P = 0.
__device__ void converter(WindowSmem& sm, const WindowParams& p, int w, int lane)
{
    // Lane l takes 16-byte unit u = l % 8 of eight rows whose numbers differ in the 8-row
    // group only, so that every address is a constant away from the first. Units 4-7 go
    // with the neighbouring row: a unit becomes two of one chunk, and units u and u + 4
    // of a row would meet in the banks.
    Seg s;
    int c = 0;
    const int u = lane & 7;
    const int key0 = 64 * (w >> 1) + 4 * (w & 1) + ((lane >> 3) ^ (u >> 2));
    const uint32_t from = sw128(key0, u), to = sw128(key0, 2 * (u & 3)) + (u >> 2) * kTile,
                   to1 = sw128(key0, 2 * (u & 3) + 1) + (u >> 2) * kTile;
    SegReader segs;
    while (segs.next(sm, p, s, lane)) {
        for (int t = s.t0; t < s.t1; ++t, ++c) {
            const int vslot = c % kVStages, hslot = c % kHStages;
            await(&sm.v_full[vslot], (c / kVStages) & 1, p.err, 4, &sm.abort);
            const uint8_t* src = sm.v[vslot] + from;
            // keys [begin, end) and those below `sink` are seen
            const int k0 = block_at(s.x, t) * kBS, begin = s.x.first - p.window + 1 - k0, end = s.x.last + 1 - k0,
                      sink = p.sinks - k0;
            const bool whole = end >= kBS && (begin <= 0 || sink >= kBS);
            await(&sm.h_empty[hslot], ((c / kHStages) & 1) ^ 1, p.err, 8, &sm.abort);
            uint8_t* dst = sm.vh[hslot][0];
#pragma unroll 1
            for (int i0 = 0; i0 < 8; i0 += 4) {
                uint4 x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint4*>(src + 1024 * (i0 + i));
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = key0 + 8 * (i0 + i);
                        if (key >= end || (key < begin && key >= sink)) x[i] = make_uint4(0, 0, 0, 0);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    *reinterpret_cast<uint4*>(dst + to + 1024 * (i0 + i)) =
                        make_uint4(codes_to_half2(x[i].x & 0xFFFFu), codes_to_half2(x[i].x >> 16),
                                   codes_to_half2(x[i].y & 0xFFFFu), codes_to_half2(x[i].y >> 16));
                    *reinterpret_cast<uint4*>(dst + to1 + 1024 * (i0 + i)) =
                        make_uint4(codes_to_half2(x[i].z & 0xFFFFu), codes_to_half2(x[i].z >> 16),
                                   codes_to_half2(x[i].w & 0xFFFFu), codes_to_half2(x[i].w >> 16));
                }
            }
            // (the codes are free once the stores have them: an arrival behind the loads alone
            // let the next block's overtake them)
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.v_empty[vslot]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.h_full[hslot]);
        }
    }
}

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// The MMAs' warp; one elected thread issues. P V of a step and S of the step after next,
// which is the same warpgroup's, go one behind the other, so that the tensor core itself
// keeps them apart where they share columns. It has at most a step's work ahead, so that
// what this warp does between two steps is time that it idles, and a warp that polls takes
// issue slots from the softmax warps on its quarter of the SM, which every step waits for:
// nothing is polled (throughout, two prompts of 5000 tokens took 836 us, against 758), and
// whether the next S's operands are there is looked up ahead of the wait for P.
__device__ void mma_issuer(WindowSmem& sm, const WindowParams& p, uint32_t tmem, int lane)
{
    constexpr uint32_t kIdescS = idesc_e4m3(128, kBS, 0, 0);
    constexpr uint32_t kIdescO = idesc_f16(128, kD, 0, 1);   // P K-major in tensor memory, V MN-major
    const uint64_t q0 = smem_desc(smem_u32(sm.q), 16, 1024, kSmem128BSwizzle);
    const uint64_t k0 = smem_desc(smem_u32(sm.k[0]), 16, 1024, kSmem128BSwizzle);
    const uint64_t v0 = smem_desc(smem_u32(sm.vh[0][0]), kTile, 1024, kSmem128BSwizzle);
    Seg s;
    SegReader segs;
    uint32_t block0 = 0, step0 = 0;              // blocks and steps before the item
    auto have_k = [&](uint32_t block) { return mbar_test(&sm.k_full[block % kSStages], (block / kSStages) & 1); };
    auto await_k = [&](uint32_t block) {
        await(&sm.k_full[block % kSStages], (block / kSStages) & 1, p.err, 16, &sm.abort);
        __syncwarp();
        tc_fence_after();
    };
    auto await_h = [&](uint32_t block) {
        await(&sm.h_full[block % kHStages], (block / kHStages) & 1, p.err, 32, &sm.abort);
    };
    auto await_p = [&](uint32_t step) {
        await(&sm.p_full[step & 1], (step >> 1) & 1, p.err, 32, &sm.abort);
        __syncwarp();
        tc_fence_after();
    };
    // by one thread
    auto issue_s = [&](uint32_t w, uint32_t block, uint32_t tile) {
        const uint64_t qd = q0 + tile * (kTile / 16), kd = k0 + (block % kKStages) * (kTile / 16);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) umma_e4m3(tmem + kSCol + kBS * w, qd + 2 * kk, kd + 2 * kk, kIdescS, kk);
        umma_commit(&sm.s_full[w]);
    };
    auto issue_pv = [&](uint32_t w, uint32_t block, bool begin, Span span) {
        const uint64_t vd = v0 + (block % kHStages) * (2 * kTile / 16);
        // 16 keys: 8 columns of P, 2048 bytes of V
        auto add = [&](int kk, bool more) {
            umma_f16_ta(tmem + kD * w, tmem + kSCol + kBS * w + 8 * kk, vd + 128 * kk, kIdescO, more ? 1u : 0u);
        };
        if (__builtin_expect(span.b - span.a == kBS / kChunk, 1)) {
#pragma unroll
            for (int kk = 0; kk < kBS / 16; ++kk) add(kk, !begin || kk > 0);
        } else {
#pragma unroll 1
            for (int kk = 2 * span.a; kk < 2 * span.b; ++kk) add(kk, !begin || kk > 2 * span.a);
        }
    };
#pragma unroll 1
    for (int item = 0; segs.next(sm, p, s, lane); ++item) {
        const int nb = s.t1 - s.t0;
        auto span_of = [&](int i) {
            Span span = {0, kBS / kChunk};
            if (__builtin_expect(s.t0 + i <= s.x.sink_blocks || s.t0 + i + 1 == s.x.blocks, 0)) span = chunks_of(p, s.x, s.t0 + i);
            return span;
        };
        await(&sm.q_full, item & 1, p.err, 16, &sm.abort);
        await_k(block0);
        const bool pair = s.x.rows > kTileRows;
        const int steps = pair ? 2 * nb : nb;
        // S of step k, and what its end frees
        auto issue_step = [&](int k) {
            const uint32_t block = block0 + (pair ? k >> 1 : k);
            const bool block_ends = !pair || (k & 1);
            issue_s((step0 + k) & 1, block, pair ? k & 1 : 0);
            if (block_ends) umma_commit(&sm.k_empty[block % kKStages]);
            if (k + 1 == steps) umma_commit(&sm.q_empty);
        };
        if (elect_one()) issue_step(0);
        __syncwarp();
        if (steps > 1) {
            if (!pair) await_k(block0 + 1);
            if (elect_one()) issue_step(1);
            __syncwarp();
        }
#pragma unroll 1
        for (int k = 0; k < steps; ++k) {
            const int i = pair ? k >> 1 : k;
            const uint32_t w = (step0 + k) & 1, block = block0 + i, next = block + (pair ? 1 : 2);
            const bool second = pair && (k & 1);     // (the first has seen K and V)
            const bool more = k + 2 < steps;
            const Span span = span_of(i);
            const bool ahead = more && (second || __all_sync(0xffffffffu, have_k(next)));
            if (!second) await_h(block);
            await_p(step0 + k);
            if (elect_one()) {
                issue_pv(w, block, k < 2, span);
                if (!pair || second) umma_commit(&sm.h_empty[block % kHStages]);
                if (!more) umma_commit(&sm.o_full[w]);
                if (ahead) issue_step(k + 2);
            }
            __syncwarp();
            if (more && !ahead) {
                await_k(next);
                if (elect_one()) issue_step(k + 2);
                __syncwarp();
            }
        }
        step0 += steps;
        block0 += nb;
    }
    __syncwarp();
    if (elect_one()) {
        umma_commit(&sm.drain);
        mbar_wait_drain(&sm.drain, 0, p.err, 512);
    }
    __syncwarp();
}

__device__ __forceinline__ void cp_async16_at(uint32_t dst, const void* src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Q rows (128-byte swizzled), q_scale and v_scale of each item.
__device__ void q_loader(WindowSmem& sm, const WindowParams& p, int lane)
{
    Seg s;
    SegReader segs;
    const int step_t = 4 / p.G, step_h = 4 - step_t * p.G;
    const int64_t step = (static_cast<int64_t>(step_t) * p.NQ + step_h) * kD, wrap = static_cast<int64_t>(p.NQ - p.G) * kD;
    for (int item = 0; segs.next(sm, p, s, lane); ++item) {
        const int buf = item & 1;
        if (!__all_sync(0xffffffffu, await(&sm.q_empty, (item & 1) ^ 1, p.err, 1024, &sm.abort))) break;
        // row r of the item: rest + r of the heads from token t on
        const int period = kTileRows / copies_of(s.x.rows), t = tokens_of(p, s.x.row0), rest = s.x.row0 - t * p.G;
        const int64_t first = static_cast<int64_t>(s.tok + t) * p.NQ + s.h * p.G;
        auto row_of = [&](int of) {
            const uint32_t n = rest + of, d = (n * p.g_mul) >> 22;
            return static_cast<int>(d * p.NQ + n - d * p.G);
        };
        // Four rows at once, a unit of 16 bytes a lane: the next four lie step further, or
        // that and wrap where the lane's row is another token's. (A tile's rows or two's, or
        // the copies of fewer.)
        const int l3 = lane >> 3, u = lane & 7, once = s.x.rows > kTileRows ? kItemRows : period;
        const uint32_t to = smem_u32(sm.q) + 128 * l3 + 16 * (u ^ l3);
#pragma unroll 1
        for (int r0 = 0; r0 < max(once, kTileRows); r0 += once) {
            const uint8_t* src = p.q + (first + row_of(l3)) * kD + 16 * u;
            int h = rest + l3;
            h -= static_cast<int>((static_cast<uint32_t>(h) * p.g_mul) >> 22) * p.G;
#pragma unroll 2
            for (int r = 0; r < once; r += 4) {
                const bool in = r + l3 < s.x.rows;
                cp_async16_at(to + 128 * (r0 + r) ^ (16 * (r & 4)), in ? src : p.q, in ? 16 : 0);
                src += step;
                h += step_h;
                if (h >= p.G) {
                    h -= p.G;
                    src += wrap;
                }
            }
        }
#pragma unroll 1
        for (int r = lane; r < max(once, kTileRows); r += 32) {
            const int of = r & (once - 1);
            cp_async4(&sm.qs[buf][r], p.q_scale + first + (of < s.x.rows ? row_of(of) : 0), 4);
        }
        cp_async16(&sm.vs[buf][4 * lane], p.v_scale + (static_cast<int64_t>(s.b) * p.NKV + s.h) * kD + 4 * lane, 16);
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_full);
    }
}

// bits 0 .. n - 1 of 32
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1); }

// Columns [0, 16 n) of tensor memory times f: floats, or (halves) pairs of FP16.
__device__ __forceinline__ void scale_columns(uint32_t taddr, int n, float f, bool halves)
{
#pragma unroll 1
    for (int c = 0; c < n; ++c) {
        float o[16];
        uint32_t y[16];
        tmem_ld16(taddr + 16 * c, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            y[i] = __float_as_uint(o[i] * f);
            if (halves) {
                const uint32_t u = __float_as_uint(o[i]);
                const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&u));
                y[i] = half2_bits(x.x * f, x.y * f);
            }
        }
        tmem_st16(taddr + 16 * c, y);
    }
    tmem_wait_st();
}

// Warpgroup w: the thread of row 32 q4 + lane of its tile.
__device__ void softmax(WindowSmem& sm, const WindowParams& p, uint32_t tmem, int w, int q4, int lane)
{
    const int trow = 32 * q4 + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * q4) << 16;
    const uint32_t O = tmem + lanes + kD * w, S = tmem + lanes + kSCol + kBS * w;
    Seg s;
    uint32_t step0 = 0, turn = 0, outs = 0;  // steps of all warpgroups before the item, own ones, items with own ones
    int block0 = 0;                          // blocks before the item
    SegReader segs;
    uint32_t joins = 0;
    // all softmax threads (a barrier with a limit, like every wait)
    auto sync_all = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.joined);
        await(&sm.joined, joins & 1, p.err, 8192, &sm.abort);
        ++joins;
        __syncwarp();
        tc_fence_after();
    };
#pragma unroll 1
    for (int item = 0; segs.next(sm, p, s, lane); ++item) {
        const bool pair = s.x.rows > kTileRows;
        const int nb = s.t1 - s.t0, steps = pair ? 2 * nb : nb;
        const int k_first = (w ^ static_cast<int>(step0)) & 1;   // this warpgroup's first step of the item
        // the row in the item, and this thread's chunks of a block's keys
        const int copies = copies_of(s.x.rows), row_off = pair ? kTileRows * k_first : 0;
        const int row = (trow & (kTileRows / copies - 1)) + row_off;
        const int c0 = trow / (kTileRows / copies) * (kBS / kChunk / copies), c1 = c0 + kBS / kChunk / copies;
        const bool live = row < s.x.rows, warp_live = row - lane < s.x.rows;
        const int pos = s.x.first + tokens_of(p, s.x.row0 + (live ? row : 0)) - tokens_of(p, s.x.row0);
        await(&sm.q_full, item & 1, p.err, 64, &sm.abort);
        float rs = live ? sm.qs[item & 1][trow + row_off] * p.scale_log2 : 1.0f;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_empty);
        // the maximum of S k_scale has to stay one under a negative scale: S changes sign
        const bool flip = rs < 0.0f, any_flip = __any_sync(0xffffffffu, flip);
        rs = fabsf(rs);
        if (rs < 1.17549435e-38f) rs = 1.17549435e-38f;       // (-inf times it stays -inf; a NaN stays, too)
        float m = -INFINITY, l = 0.0f, nref = 0.0f, limit = -1.0f;   // (nref: 7 - m, or 0; the first chunk sets m)
#pragma unroll 1
        for (int k = k_first; k < steps; k += 2, ++turn) {
            const int t = pair ? k >> 1 : k;
            const uint32_t at = block0 + t;
            if (__builtin_expect(!warp_live, 0)) {   // a warp without rows keeps the others company
                await(&sm.s_full[w], turn & 1, p.err, 64, &sm.abort);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full[w]);
                continue;
            }
            // (all that does not wait for S; behind it, it costs 6% of a prompt)
            await(&sm.k_full[at % kSStages], (at / kSStages) & 1, p.err, 64, &sm.abort);
            const float4* ks = reinterpret_cast<const float4*>(sm.ks[at % kSStages]);
            // keys up to the row's own (end), and of those its window's (from begin) and the
            // sinks (below sink); whether any row does not see all
            const int k0 = block_at(s.x, s.t0 + t) * kBS, sink = p.sinks - k0;
            const bool part_seen = s.x.first - k0 < kBS - 1 || (s.x.last - k0 >= p.window && sink < kBS);
            const int end = pos + 1 - k0, begin = end - p.window;
            const Span span = chunks_of(p, s.x, s.t0 + t);
            const int ca = max(c0, span.a), cb = min(c1, span.b);
            await(&sm.s_full[w], turn & 1, p.err, 64, &sm.abort);
            __syncwarp();
            tc_fence_after();
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int c = ca; c < cb; ++c) {
                float v[kChunk];
                tmem_ld32(S + kChunk * c, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < kChunk / 4; ++i) {
                    const float4 k4 = ks[kChunk / 4 * c + i];
                    const float2 a = __fmul2_rn(make_float2(v[4 * i], v[4 * i + 1]), make_float2(k4.x, k4.y));
                    const float2 b = __fmul2_rn(make_float2(v[4 * i + 2], v[4 * i + 3]), make_float2(k4.z, k4.w));
                    v[4 * i] = a.x;
                    v[4 * i + 1] = a.y;
                    v[4 * i + 2] = b.x;
                    v[4 * i + 3] = b.y;
                }
                if (__builtin_expect(part_seen || any_flip, 0)) {
                    const uint32_t see = bits_below(end - kChunk * c) &
                                         (~bits_below(begin - kChunk * c) | bits_below(sink - kChunk * c));
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) v[i] = !((see >> i) & 1) ? -INFINITY : (flip ? -v[i] : v[i]);
                }
                // P = 2^(x - m + 7). Its sum tells whether all are inside FP16; if not, or where
                // there is no m yet, the maximum is looked up and it is done again.
                uint32_t hp[kChunk / 2];
                float2 part;
                float rx = rs;
                bool again = false;
#pragma unroll 1
                for (;;) {
                    const float2 rs2 = make_float2(rx, rx), ref2 = make_float2(nref, nref);
                    part = make_float2(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < kChunk / 2; ++i) {
                        float2 x = __ffma2_rn(make_float2(v[2 * i], v[2 * i + 1]), rs2, ref2);
                        x.x = ex2(x.x);
                        x.y = ex2(x.y);
                        part = __fadd2_rn(part, x);
                        hp[i] = half2_bits(x.x, x.y);
                    }
                    if (__builtin_expect(again || __all_sync(0xffffffffu, part.x + part.y <= limit), 1)) break;
                    again = true;
                    float mx = fmaxf(v[0], v[1]);
#pragma unroll
                    for (int i = 2; i < kChunk; i += 2) mx = max3(mx, v[i], v[i + 1]);
                    mx *= rs;
                    const bool raise = mx > m + kRaise;
                    if (__any_sync(0xffffffffu, raise)) {
                        const float f = raise ? ex2(m - mx) : 1.0f;      // (0 while m is -inf)
                        m = raise ? mx : m;
                        l *= f;
                        sum = make_float2(sum.x * f, sum.y * f);
                        // (this step's S is complete, so the last step's P V is)
                        if (k > k_first) scale_columns(O, kD / 16, f, false);
                        // P of the block's keys so far
                        tmem_wait_st();
                        if (c > ca) scale_columns(S + kChunk / 2 * ca, c - ca, f, true);
                    }
                    // Past 2^22 the rounding of m is no longer small beside the exponents, which
                    // take the products unrounded (one too large by 1 leaves FP16): there they are
                    // rounded as m is, every time.
                    const bool none = m == -INFINITY, big = fabsf(m) > 0x1p22f && !none;
                    nref = none ? 0.0f : kShift - m;
                    limit = none || big ? -1.0f : kLimit;
                    if (__any_sync(0xffffffffu, big)) {
                        const float f = big ? rs : 1.0f;
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) v[i] *= f;
                        rx = big ? 1.0f : rs;
                    }
                }
                sum = __fadd2_rn(sum, part);
                tmem_st16(S + kChunk / 2 * c, hp);
            }
            // the other copies' keys
            if (copies > 1) {
                uint32_t zero[kChunk / 2];
#pragma unroll
                for (int i = 0; i < kChunk / 2; ++i) zero[i] = 0;
#pragma unroll 1
                for (int c = span.a; c < span.b; ++c)
                    if (c < c0 || c >= c1) tmem_st16(S + kChunk / 2 * c, zero);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full[w]);
            l += sum.x + sum.y;
        }
        // ---- the item's (or its part's) output ----
        const bool whole = s.t0 == 0 && s.t1 == s.x.blocks;
        float* const part = part_of(p, blockIdx.x, s.first_of_run);
        float* const part_ml = part + static_cast<int64_t>(p.part_rows) * kD;
        // (behind all that does not need O)
        auto o_complete = [&] {
            if (k_first < steps) {
                await(&sm.o_full[w], outs & 1, p.err, 128, &sm.abort);
                ++outs;
            }
            __syncwarp();
            tc_fence_after();
        };
        if (pair) {
            const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
            const int64_t at = q_row(p, s.tok, s.h, s.x.row0 + (live ? row : 0)) * kD;
            o_complete();
#pragma unroll 1
            for (int c = 0; c < kD && warp_live; c += 16) {
                __syncwarp();                // (rows behind the last one store nothing)
                float o[16];
                tmem_ld16(O + c, o);
                tmem_wait_ld();
                if (!live) continue;
                if (whole) {
                    const float4* vs = reinterpret_cast<const float4*>(sm.vs[item & 1] + c);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float4 a = vs[2 * i], e = vs[2 * i + 1];
                        const float* x = o + 8 * i;
                        const __nv_bfloat162 y0 = __floats2bfloat162_rn(x[0] * inv * a.x, x[1] * inv * a.y);
                        const __nv_bfloat162 y1 = __floats2bfloat162_rn(x[2] * inv * a.z, x[3] * inv * a.w);
                        const __nv_bfloat162 y2 = __floats2bfloat162_rn(x[4] * inv * e.x, x[5] * inv * e.y);
                        const __nv_bfloat162 y3 = __floats2bfloat162_rn(x[6] * inv * e.z, x[7] * inv * e.w);
                        reinterpret_cast<uint4*>(p.out + at + c)[i] = make_uint4(
                            *reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1),
                            *reinterpret_cast<const uint32_t*>(&y2), *reinterpret_cast<const uint32_t*>(&y3));
                    }
                } else {
                    float4* dst = reinterpret_cast<float4*>(part + row * kD + c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
            }
            if (!whole && live) {
                part_ml[row] = m;
                part_ml[p.part_rows + row] = l;
            }
        } else {
            // the sums of every row: over the warpgroups in registers (their O lie in the same
            // lanes), over the copies through shared memory, 32 channels of the 128 lanes or
            // 64 of the 64 that count at a time
            sm.m[w * kTileRows + trow] = m;
            sm.l[w * kTileRows + trow] = l;
            sync_all();
            const int period = kTileRows / copies, narrow = s.x.rows <= 32 ? 1 : 0;
            float mf = -INFINITY, lt = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < 2 * copies) mf = fmaxf(mf, sm.m[(trow + i * period) & (2 * kTileRows - 1)]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int from = (trow + i * period) & (2 * kTileRows - 1);
                if (i < 2 * copies && sm.l[from] != 0.0f)
                    lt += sm.l[from] * (sm.m[from] == mf ? 1.0f : ex2(sm.m[from] - mf));
            }
            // (nothing summed, perhaps nothing written; a NaN has to reach the output)
            const bool has0 = sm.l[trow] != 0.0f, has1 = sm.l[kTileRows + trow] != 0.0f;
            const float m0 = sm.m[trow], m1 = sm.m[kTileRows + trow];
            const float f0 = m0 == mf ? 1.0f : ex2(m0 - mf), f1 = m1 == mf ? 1.0f : ex2(m1 - mf);
            if (w == 0 && trow < period) {
                sm.inv[trow] = lt == 0.0f ? 0.0f : __fdiv_rn(1.0f, lt);
                if (!whole && live) {
                    part_ml[row] = mf;
                    part_ml[p.part_rows + row] = lt;
                }
            }
            // (both warpgroups' O, which every thread reads)
            o_complete();
            sync_all();
            // a lane's units of four channels (8 or 16 of them), and its place in the buffer
            const int units = 8 << narrow, lane_at = narrow ? 32 * (q4 >> 1) + lane : trow;
            const int tid = w * kTileRows + trow, j = tid & (units - 1);
#pragma unroll 1
            for (int c = 0; c < kD; c += 4 * units) {
#pragma unroll 1
                for (int u = w * units / 2; u < (w + 1) * units / 2 && !(narrow && (q4 & 1)); u += 4) {
                    float x[16], y[16];
                    tmem_ld16(tmem + lanes + c + 4 * u, x);
                    tmem_ld16(tmem + lanes + kD + c + 4 * u, y);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = (has0 ? x[i] * f0 : 0.0f) + (has1 ? y[i] * f1 : 0.0f);
#pragma unroll
                    for (int i = 0; i < 4; ++i)      // (a lane's units begin at another place each)
                        sm.join[lane_at * units + ((u + i + lane_at) & (units - 1))] =
                            make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                }
                sync_all();
#pragma unroll 1
                for (int r = tid >> (3 + narrow); r < s.x.rows; r += 256 >> (3 + narrow)) {
                    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (i >= copies) break;
                        const int from = r + (narrow ? 32 : period) * i;
                        const float4 x = sm.join[from * units + ((j + from) & (units - 1))];
                        sum = make_float4(sum.x + x.x, sum.y + x.y, sum.z + x.z, sum.w + x.w);
                    }
                    if (whole) {
                        const float inv = sm.inv[r];
                        const float4 vs = *reinterpret_cast<const float4*>(sm.vs[item & 1] + c + 4 * j);
                        const __nv_bfloat162 y0 = __floats2bfloat162_rn(sum.x * inv * vs.x, sum.y * inv * vs.y);
                        const __nv_bfloat162 y1 = __floats2bfloat162_rn(sum.z * inv * vs.z, sum.w * inv * vs.w);
                        *reinterpret_cast<uint2*>(p.out + q_row(p, s.tok, s.h, s.x.row0 + r) * kD + c + 4 * j) =
                            make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
                    } else {
                        *reinterpret_cast<float4*>(part + r * kD + c + 4 * j) = sum;
                    }
                }
                sync_all();
            }
        }
        // (the other's m and l are read until here; the last barrier was behind them)
        tc_fence_before();
        __syncwarp();
        step0 += steps;
        block0 += nb;
    }
}

// What the joining kernel has to know of the item at the begin of this CTA's run. Block
// t of an item that begins at `base` is at position base + kItemCost + u (t + 1) - 1, u
// its steps; a run holds at least two positions, so the runs c0 to c1 with its first and
// its last block have one each.
__device__ void describe_cut(WindowSmem& sm, const WindowParams& p, const Run& run, uint32_t total, uint32_t ctas, int lane)
{
    const int c = blockIdx.x;
    Cut cut = {};
    if (run.pos < run.hi && run.pos > run.base) {
        const Item x = item_of(p, sm.pos[run.b], sm.rows[run.b], run.i);
        const int u = steps_a_block(x.rows);
        const int c0 = cta_of(total, run.base + kItemCost + u - 1, ctas);
        const int c1 = cta_of(total, run.base + weight_of(x) - 1, ctas);
        if (c == c0 + 1 && c0 < c1) {
            cut.b = run.b;
            cut.h = run.h;
            cut.row0 = x.row0;
            cut.rows = x.rows;
            cut.tok0 = sm.tok[run.b];
            cut.c0 = c0;
            cut.c1 = c1;
            cut.slot0 = 2 * c0 + (run_begin(total, c0, ctas) >= run.base ? 0 : 1);
        }
    }
    if (lane == 0) p.cuts[c] = cut;
}

// Zeros for the tokens that see nothing: those before, between and behind the sequences'
// live ones. Token t is CTA t % gridDim's, whose scheduling warp writes it while the others
// are at the run's last items: a refused chunk of 5000 tokens beside 32 decoding requests of
// 96 heads (123 MB) takes the call from 31 us to 46, and took it to 1884 when one CTA wrote a
// sequence's, ahead of its items.
__device__ void zero_rows(const WindowSmem& sm, const WindowParams& p, int lane)
{
    const int ctas = gridDim.x;
    for (int g0 = 0; g0 <= p.B; g0 += 32) {
        const int g = g0 + lane;
        int at = 0, end = 0;                 // between sequence g - 1's live tokens and sequence g's
        if (g <= p.B) {
            at = g > 0 ? sm.tok[g - 1] + tokens_of(p, sm.rows[g - 1]) : min(max(__ldg(p.cu), 0), p.T);
            end = g < p.B ? sm.tok[g] : min(max(__ldg(p.cu + p.B), 0), p.T);
        }
        for (uint32_t some = __ballot_sync(0xffffffffu, at < end); some != 0; some &= some - 1) {
            const int a = __shfl_sync(0xffffffffu, at, __ffs(some) - 1), e = __shfl_sync(0xffffffffu, end, __ffs(some) - 1);
            const int64_t first = static_cast<int64_t>(a) + (static_cast<int>(blockIdx.x) + ctas - a % ctas) % ctas;
            for (int64_t t = first; t < e; t += ctas) {
                uint4* dst = reinterpret_cast<uint4*>(p.out + t * p.NQ * kD);
                for (int j = lane; j < p.NQ * (kD / 8); j += 32) dst[j] = make_uint4(0, 0, 0, 0);
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1)
    window_attention_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                            const __grid_constant__ WindowParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uintptr_t raw = reinterpret_cast<uintptr_t>(smem_raw);
    WindowSmem& sm = *reinterpret_cast<WindowSmem*>(smem_raw + ((1024u - (raw & 1023u)) & 1023u));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < kSStages; ++i) mbar_init(&sm.k_full[i], 33);
        for (int i = 0; i < kKStages; ++i) mbar_init(&sm.k_empty[i], 1);
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_empty[i], kConvWarps);
        }
        for (int i = 0; i < kHStages; ++i) {
            mbar_init(&sm.h_full[i], kConvWarps);
            mbar_init(&sm.h_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_full[i], 4);
            mbar_init(&sm.o_full[i], 1);
        }
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(&sm.seg_full[i], 1);
            mbar_init(&sm.seg_empty[i], kSegReaders);
        }
        mbar_init(&sm.joined, 8);
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 1 + 8);
        mbar_init(&sm.drain, 1);
        sm.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(&sm.tmem, kTmemCols);
    grid_launch_dependents();   // (the joining kernel waits for this one's end)
    int group;
    const uint32_t total = build_schedule(sm, p, tid, group);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    // runs of kMinRun positions at least
    const uint32_t ctas = max(1u, min(static_cast<uint32_t>(p.ctas), total / kMinRun));

    if (warp < kProdWarp) {
        softmax(sm, p, tmem, warp >> 2, warp & 3, lane);
    } else if (warp == kProdWarp) {
        producer(sm, p, &tk, &tv, lane);
    } else if (warp == kMmaWarp) {
        mma_issuer(sm, p, tmem, lane);
    } else if (warp == kQWarp) {
        q_loader(sm, p, lane);
    } else if (warp == kSegWarp) {
        Run run = {};
        if (blockIdx.x < ctas && total > 0)
            run = locate(sm, p, group, run_begin(total, blockIdx.x, ctas), run_begin(total, blockIdx.x + 1, ctas));
        scheduler(sm, p, run, lane);
        describe_cut(sm, p, run, total, ctas, lane);
        zero_rows(sm, p, lane);
    } else {
        converter(sm, p, warp - kConvWarp, lane);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the parts of the items that a run's end cut: CTA (c, y) takes the item whose
// first block run c has and whose last one a later run, a warp two rows of it and four
// parts at once, all their loads in flight together.
constexpr int kJoinWarps = 4, kJoinRows = 2, kJoinParts = 4;

__global__ void __launch_bounds__(kJoinWarps * 32) window_join_kernel(const WindowParams p)
{
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int4 a = *reinterpret_cast<const int4*>(p.cuts + blockIdx.x + 1);
    const int4 z = *(reinterpret_cast<const int4*>(p.cuts + blockIdx.x + 1) + 1);
    const int h = a.x, item0 = a.y, rows = a.z, tok0 = a.w, c0 = z.x, c1 = z.y, slot0 = z.z, b = z.w;
    const int row0 = (blockIdx.y * kJoinWarps + (threadIdx.x >> 5)) * kJoinRows;
    if (row0 >= rows) return;
    const int64_t slot_floats = static_cast<int64_t>(p.part_rows) * (kD + 2);
    // O's part of run c (its rows begin there), m and l behind the rows
    auto part = [&](int c) { return p.part + (c == c0 ? slot0 : 2 * c) * slot_floats; };
    const float4 v =
        __ldg(reinterpret_cast<const float4*>(p.v_scale + (static_cast<int64_t>(b) * p.NKV + h) * kD) + lane);
    int row[kJoinRows];
    float M[kJoinRows], L[kJoinRows];
    float4 o[kJoinRows];
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) {
        row[r] = min(row0 + r, rows - 1);
        M[r] = -INFINITY;
        L[r] = 0.0f;
        o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // in order, with a running maximum, so that no load waits for another
#pragma unroll 1
    for (int c = c0; c <= c1; c += kJoinParts) {
        float m[kJoinParts][kJoinRows], l[kJoinParts][kJoinRows];
        float4 x[kJoinParts][kJoinRows];
#pragma unroll
        for (int i = 0; i < kJoinParts; ++i) {
            const float* q = part(min(c + i, c1));
            const float* ml = q + static_cast<int64_t>(p.part_rows) * kD;
#pragma unroll
            for (int r = 0; r < kJoinRows; ++r) {
                m[i][r] = c + i <= c1 ? ml[row[r]] : -INFINITY;
                l[i][r] = c + i <= c1 ? ml[p.part_rows + row[r]] : 0.0f;
                x[i][r] = reinterpret_cast<const float4*>(q + row[r] * kD)[lane];
            }
        }
#pragma unroll
        for (int i = 0; i < kJoinParts; ++i) {
#pragma unroll
            for (int r = 0; r < kJoinRows; ++r) {
                // nothing seen in this part. (Where all scores are NaN the maximum is -inf as
                // well, and the sum NaN: that has to reach the output.)
                if (l[i][r] == 0.0f) continue;
                const float mn = fmaxf(M[r], m[i][r]);
                const float f = M[r] == mn ? 1.0f : ex2(M[r] - mn), g = m[i][r] == mn ? 1.0f : ex2(m[i][r] - mn);
                M[r] = mn;
                L[r] = L[r] * f + l[i][r] * g;
                o[r].x = o[r].x * f + x[i][r].x * g;
                o[r].y = o[r].y * f + x[i][r].y * g;
                o[r].z = o[r].z * f + x[i][r].z * g;
                o[r].w = o[r].w * f + x[i][r].w * g;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) {
        if (row0 + r >= rows) break;
        const float inv = L[r] == 0.0f ? 0.0f : __fdiv_rn(1.0f, L[r]);
        const __nv_bfloat162 y0 = __floats2bfloat162_rn(o[r].x * inv * v.x, o[r].y * inv * v.y);
        const __nv_bfloat162 y1 = __floats2bfloat162_rn(o[r].z * inv * v.z, o[r].w * inv * v.w);
        reinterpret_cast<uint2*>(p.out + q_row(p, tok0, h, item0 + row[r]) * kD)[lane] =
            make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
    }
}

// rows of the largest item, a multiple of 64 so that parts start on 256 bytes
int part_rows(int max_tokens, int G)
{
    const int64_t r = static_cast<int64_t>(max_tokens) * G;
    return r >= kItemRows ? kItemRows : static_cast<int>((r + 63) / 64 * 64);
}

pa_status check_shape(const char* name, int max_tokens, int NQ, int NKV, int D)
{
    PA_REQUIRE(max_tokens > 0 && NQ > 0 && NKV > 0 && D > 0, PA_ERR_INVALID,
               "%s: empty or negative shape (max_tokens=%d NQ=%d NKV=%d D=%d)", name, max_tokens, NQ, NKV, D);
    PA_REQUIRE(NQ % NKV == 0, PA_ERR_INVALID, "%s: NQ %d is not a multiple of NKV %d", name, NQ, NKV);
    PA_REQUIRE(D == kD, PA_ERR_UNSUPPORTED, "%s: head size %d (only 128 is built)", name, D);
    PA_REQUIRE(NQ / NKV <= kMaxGroup, PA_ERR_UNSUPPORTED, "%s: %d query heads per kv head (at most %d)", name,
               NQ / NKV, kMaxGroup);
    return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_fp8_window_attention_workspace_size(int max_tokens, int NQ, int NKV, int D, size_t* bytes)
{
    const char* name = "pa_fp8_window_attention_workspace_size";
    PA_REQUIRE(bytes, PA_ERR_NULLPTR, "%s: bytes is NULL", name);
    const pa_status st = check_shape(name, max_tokens, NQ, NKV, D);
    if (st != PA_OK) return st;
    *bytes = kPartOff + static_cast<size_t>(kMaxCtas) * 2 * part_rows(max_tokens, NQ / NKV) * (kD + 2) * sizeof(float);
    return PA_OK;
}

extern "C" pa_status pa_fp8_window_attention(const void* q, const float* q_scale, const void* k_cache,
                                             const float* k_scale, const void* v_cache, const float* v_scale,
                                             const int32_t* block_table, const int32_t* kv_act_seqs,
                                             const int32_t* cu_tokens, void* out, int B, int64_t num_tokens,
                                             int max_tokens, int NQ, int NKV, int D, int block_size,
                                             int64_t num_blocks, int max_blocks_per_seq, int layout, int64_t window,
                                             int64_t sinks, float softmax_scale, void* workspace,
                                             size_t workspace_bytes, void* stream)
{
    const char* name = "pa_fp8_window_attention";
    PA_REQUIRE(B >= 0 && num_tokens >= 0, PA_ERR_INVALID, "%s: negative size", name);
    const bool none = B == 0 || num_tokens == 0;
    // (tensors of no sequences or tokens may have no address)
    PA_REQUIRE(k_cache && k_scale && v_cache &&
                   (none || (q && q_scale && v_scale && block_table && kv_act_seqs && cu_tokens && out)),
               PA_ERR_NULLPTR, "%s: NULL tensor pointer", name);
    const pa_status ps = check_shape(name, max_tokens, NQ, NKV, D);
    if (ps != PA_OK) return ps;
    size_t need = 0;
    pa_fp8_window_attention_workspace_size(max_tokens, NQ, NKV, D, &need);
    PA_REQUIRE(num_blocks > 0 && max_blocks_per_seq > 0 && block_size > 0, PA_ERR_INVALID,
               "%s: empty cache or block table", name);
    PA_REQUIRE(block_size == kBS, PA_ERR_UNSUPPORTED, "%s: block_size %d (only 128 is built)", name, block_size);
    PA_REQUIRE(layout == PA_LAYOUT_BSND || layout == PA_LAYOUT_BNBD, PA_ERR_INVALID, "%s: unknown layout %d", name,
               layout);
    PA_REQUIRE(window >= 0 && sinks >= 0, PA_ERR_INVALID, "%s: negative window or sinks", name);
    PA_REQUIRE(std::isfinite(softmax_scale), PA_ERR_INVALID, "%s: softmax_scale not finite", name);
    PA_REQUIRE(B <= kMaxB, PA_ERR_UNSUPPORTED, "%s: batch %d > %d", name, B, kMaxB);
    PA_REQUIRE(max_blocks_per_seq < (1 << 24) / kBS, PA_ERR_UNSUPPORTED,
               "%s: block table of %d blocks, 2^24 positions or more", name, max_blocks_per_seq);
    PA_REQUIRE(num_blocks <= 0x7FFFFFFF / kBS / NKV, PA_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 cache rows", name);
    PA_REQUIRE(num_tokens <= 0x7FFFFFFF / NQ, PA_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 query rows", name);
    PA_REQUIRE(aligned16(q) && aligned16(k_cache) && aligned16(v_cache) && aligned16(v_scale) && aligned16(out),
               PA_ERR_INVALID, "%s: q, the caches, v_scale and out must be 16-byte aligned", name);
    for (const void* x : {static_cast<const void*>(q_scale), static_cast<const void*>(k_scale),
                          static_cast<const void*>(block_table), static_cast<const void*>(kv_act_seqs),
                          static_cast<const void*>(cu_tokens)})
        PA_REQUIRE((reinterpret_cast<uintptr_t>(x) & 3u) == 0, PA_ERR_INVALID,
                   "%s: q_scale, k_scale, block_table, kv_act_seqs and cu_tokens must be 4-byte aligned", name);
    // (positions lie below 2^24)
    constexpr int64_t kAll = 1 << 24;
    const int win = static_cast<int>(window == 0 ? kAll : std::min(window, kAll));
    const int first = static_cast<int>(std::min(sinks, kAll));
    // the schedule counts steps in 32 bits
    const int G = NQ / NKV;
    const int64_t items = (num_tokens * G + kItemRows - 1) / kItemRows + B;
    PA_REQUIRE(items * NKV <= 0xFFFFFFFFll / (2 * max_blocks_per_seq + kItemCost), PA_ERR_UNSUPPORTED,
               "%s: tokens * heads * max_blocks_per_seq too large for the 32-bit schedule", name);
    if (none) return PA_OK;
    PA_REQUIRE(workspace && workspace_bytes >= need, PA_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", name,
               workspace ? workspace_bytes : static_cast<size_t>(0), need);
    PA_REQUIRE((reinterpret_cast<uintptr_t>(workspace) & 255u) == 0, PA_ERR_INVALID,
               "%s: workspace must be 256-byte aligned", name);
    // every CTA reads while others already write
    struct Range { const void* at; uint64_t bytes; };
    const uint64_t codes = static_cast<uint64_t>(num_tokens) * NQ * kD, cache = static_cast<uint64_t>(num_blocks) * kBS * NKV * kD;
    const Range in[] = {{q, codes}, {q_scale, codes / kD * 4}, {k_cache, cache}, {k_scale, cache / kD * 4},
                        {v_cache, cache}, {v_scale, 4ull * B * NKV * kD}, {block_table, 4ull * B * max_blocks_per_seq},
                        {kv_act_seqs, 4ull * B}, {cu_tokens, 4ull * (B + 1)}};
    for (const Range& i : in)
        PA_REQUIRE(!overlap(out, 2 * codes, i.at, i.bytes), PA_ERR_INVALID, "%s: out overlaps an input", name);
    const int sms = device_sm_count();
    PA_REQUIRE(sms > 0, PA_ERR_CUDA, "%s: cannot query the device", name);
    CUtensorMap tk, tv;
    const uint64_t inner = layout == PA_LAYOUT_BSND ? static_cast<uint64_t>(NKV) * kD : kD;
    const uint64_t rows = static_cast<uint64_t>(num_blocks) * kBS * (layout == PA_LAYOUT_BNBD ? NKV : 1);
    pa_status st = make_cache_map(&tk, k_cache, inner, rows);
    if (st != PA_OK) return st;
    st = make_cache_map(&tv, v_cache, inner, rows);
    if (st != PA_OK) return st;

    uint8_t* ws = static_cast<uint8_t*>(workspace);
    WindowParams p;
    p.q = static_cast<const uint8_t*>(q);
    p.q_scale = q_scale;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.bt = block_table;
    p.act = kv_act_seqs;
    p.cu = cu_tokens;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.err = reinterpret_cast<int*>(ws);
    p.cuts = reinterpret_cast<Cut*>(ws + kCutOff);
    p.part = reinterpret_cast<float*>(ws + kPartOff);
    p.part_rows = part_rows(max_tokens, G);
    p.B = B;
    p.T = static_cast<int>(num_tokens);
    p.max_tokens = max_tokens;
    p.NQ = NQ;
    p.NKV = NKV;
    p.G = G;
    p.g_mul = (1u << 22) / G + 1;
    p.g_inv = ~0ull / G + 1;
    p.one_item = static_cast<int64_t>(max_tokens) * G <= kItemRows;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    p.layout = layout;
    p.ctas = sms < kMaxCtas ? sms : kMaxCtas;
    p.window = win;
    p.sinks = first;
    p.scale_log2 = softmax_scale * 1.4426950408889634f;

    cudaError_t e = cudaFuncSetAttribute(window_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSmemBytes));
    PA_REQUIRE(e == cudaSuccess, PA_ERR_CUDA, "%s: smem attribute: %s", name, cudaGetErrorString(e));
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    window_attention_kernel<<<static_cast<unsigned>(p.ctas), kThreads, kSmemBytes, cs>>>(tk, tv, p);
    st = check_launch(name);
    if (st != PA_OK || p.ctas == 1) return st;
    const int most = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(max_tokens) * G, kItemRows));
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(p.ctas - 1), static_cast<unsigned>((most + kJoinWarps * kJoinRows - 1) / (kJoinWarps * kJoinRows)));
    lc.blockDim = dim3(kJoinWarps * 32);
    lc.stream = cs;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    e = cudaLaunchKernelEx(&lc, window_join_kernel, p);
    PA_REQUIRE(e == cudaSuccess, PA_ERR_CUDA, "%s: launch: %s", name, cudaGetErrorString(e));
    return PA_OK;
}
