// tree.cu -- attention of a tree of drafted tokens over the paged FP8 cache.
//
// The query rows that share a kv head are the S1 drafted tokens x the group of
// query heads: R = n G rows of sequence b, each attending to the context and
// to the drafted tokens its mask row names. Rows are taken in items of at most
// 128, one tensor tile.
//
//   S = Q_fp8 K_fp8^T                 tcgen05 kind::f8f6f4, 128 rows x 128 keys
//   x = S k_scale q_scale scale log2e, -inf where the row does not see the key
//   P = 2^(x - m + 7), L += sum P     one thread per row, FP32
//   O += FP16(P) V                    tcgen05 kind::f16, P from tensor memory
//   out = BF16(O v_scale / L)
//
// P enters the second contraction as FP16 (half a step: 2^-11) and V as the
// FP16 values of its E4M3 codes, which are exact: P in E4M3 as in
// pa_fp8_decode would be off by up to 2^-4 where few keys count. The reference
// m is the running maximum, but raised only when a block's maximum lies
// more than 2^8 above it, which spares O's rescaling in tensor memory on most;
// P then stays below 2^15, inside FP16, and a key 2^31 below the maximum still
// counts.
//
// What bounds it short of HBM is the chain from one tensor instruction to the
// next: a batch of MMAs and its commit take about 1000 clocks from the wake-up of
// the issuing warp to that of the waiting one, and each hand-over between warps
// another 50 to 100. So steps are large (a block of 128 keys, whose scores a
// thread holds in registers) and overlap: two softmax warpgroups take blocks in
// turn, each with an S and a P buffer of its own (tensor memory: O 128 columns, S
// 2 x 128, P 2 x 64), and S of a warpgroup's next block is computed while it works
// on the last. They share m, row by row: a warp decides on m for its block after
// the other warpgroup's warp has decided on the block before, and only the
// exponentials wait for that. A block then takes about 1800 clocks; HBM would
// take 1400.
//
// Measured, a pass: 4 sequences of up to 131072 keys x 5 x 96 heads over 8: 128 to
// 133 us from box to box (645 MB, 4.9 TB/s; steps of 64 keys with twice the buffers
// 147, three warpgroups 151); 16 of up to 4096 x 64: 131 us (111 GFLOP, 0.85 PFLOP/s,
// of items of 16 blocks on average); the same x 8: 31 us; 2 of up to 300 keys x 8 x 4
// heads: 10 us. Where the code lies counts: the loops' parts move against one
// another, and the same arithmetic has taken up to 16% longer.
//   warps 0-7        softmax, warpgroup k of blocks k, k + 2, .. (thread = row =
//                    tensor memory lane)
//   warp 8           K and V blocks by TMA, key scales by cp.async; tells the joining
//                    kernel about the item at the run's begin
//   warps 9, 10      issue S, issue P V
//   warp 11          Q rows and scales of the next segment
//   warps 12-15      V codes to FP16 in shared memory, zeros behind the end
//
// The items in (sequence, kv head, row tile) order are dealt to the CTAs in runs
// of equal weight: a block counts 1, an item kItemCost besides. Items that a
// run's end cuts leave FP32 partial sums, which a second kernel joins.
#include "attend.cuh"

#include <cmath>
#include <cstddef>

namespace pa {
namespace {

constexpr int kD = 128;
constexpr int kBS = 128;
constexpr int kMaxNodes = 128;
constexpr int kMaxGroup = 128;
constexpr int kMaxB = 1024;
constexpr int kMaxCtas = 192;
constexpr int kItemRows = 128;
constexpr int kTile = kBS * kD;              // bytes of a block of codes
// K blocks, V blocks as codes and as FP16, key scales. The scales' ring needs no
// barrier that says a slot is free: block i + 8 is requested once K block i + 4
// is free, i.e. its S complete; that was issued after block i + 2's had left its
// S buffer, and so after its warpgroup was done with block i.
constexpr int kKStages = 4, kVStages = 3, kHStages = 2, kSStages = 8;
// Softmax warpgroups, which take blocks in turn, each with an S and a P buffer of
// its own.
constexpr int kTurns = 2;
constexpr int kProdWarp = 4 * kTurns, kMmaWarp = kProdWarp + 1, kQWarp = kProdWarp + 3;
constexpr int kConvWarp = kProdWarp + 4, kConvWarps = 4;
constexpr int kThreads = (kConvWarp + kConvWarps) * 32;
// Registers: 512 threads start with 128 each; the softmax warpgroups, which hold
// 128 scores a thread, go up to 200 and the other two down to 56 (256 x 200 + 256
// x 56 = 512 x 128; 184 and 72 spill more and are 1% slower).
constexpr int kSoftmaxRegs = 200, kOtherRegs = 56;
constexpr uint32_t kTmemCols = 512, kSCol = 128, kPCol = kSCol + kTurns * kBS;   // O, then S, then P
constexpr float kRaise = 8.0f;               // log2 units: see the top of the file
constexpr float kShift = 7.0f;

// What an item costs besides its blocks, in blocks: the last block's softmax and
// P V, its output and the first softmax of the next item, about 10000 clocks.
// 5, 6, 7: 133, 128, 127 us on 16 sequences of up to 4096 keys (as 1 to 4096 fall
// out) x 64 drafted tokens x 96 heads over 8, 31.4, 31.7, 32.8 with 8 drafted tokens.
constexpr int kItemCost = 6;

// What the joining kernel has to know of the item at the begin of a run.
struct Cut {
    int b, h, row0, rows;                    // rows 0: nothing to join
    int c0, c1;                              // the runs that have its first and its last block
    int slot0, pad;                          // where run c0's part lies
};

// Workspace: error word, a Cut per CTA, then per CTA two partial items: O
// [rows][128], m and l [rows]. Slot 2 c is of run c's first item, slot 2 c + 1
// of its last. l = 0: the row sees nothing there.
constexpr size_t kCutOff = 256;
constexpr size_t kPartOff = kCutOff + kMaxCtas * sizeof(Cut);

struct TreeParams {
    const uint8_t* q;
    const float* q_scale;
    const float* k_scale;
    const float* v_scale;
    const int *bt, *act, *len;
    const uint8_t* mask;
    int64_t mask_stride;
    __nv_bfloat16* out;
    int* err;
    Cut* cuts;
    float* part;
    int part_rows;                           // rows of a partial item
    int B, S1, NQ, NKV, G;
    uint32_t g_mul;                          // 2^22 / G + 1: n / G = n g_mul >> 22 for n < 2^14
    int64_t num_blocks;
    int max_blocks, layout, ctas;
    int keep_l2;                             // K/V blocks serve several items
    float scale_log2;
};

struct TreeSmem {
    alignas(1024) uint8_t k[kKStages][kTile];
    alignas(1024) uint8_t v[kVStages][kTile];
    alignas(1024) uint8_t vh[kHStages][2][kTile];   // FP16, channels 0-63 and 64-127
    alignas(1024) uint8_t q[2][kTile];              // by segment parity, as qs and vs
    alignas(16) float ks[kSStages][kBS];
    alignas(16) float qs[2][kItemRows];
    alignas(16) float vs[2][kD];
    float m[kItemRows], ml[2][kTurns][kItemRows];
    uint32_t cum[kMaxB + 1];                 // weights before each sequence
    uint32_t len[kMaxB];                     // length << 8 | drafted tokens
    uint64_t k_full[kSStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
    uint64_t h_full[kHStages], h_empty[kHStages];
    uint64_t s_full[kTurns], s_free[kTurns], p_full[kTurns], o_done[kTurns], q_full[2], q_empty[2], drain[2];
    uint32_t tmem;
    int abort;
};
constexpr size_t kSmemBytes = offsetof(TreeSmem, abort) + sizeof(int) + 1024;   // (aligned by hand)
static_assert(kSmemBytes <= 232448, "tree decode shared memory over budget");

// ---- the schedule -----------------------------------------------------------------
struct Seg {
    int b, h, row0, rows;                    // the item
    int t0, t1, tiles;                       // its blocks that this run has
    bool first;                              // first of the CTA's run
};

struct Run {
    uint32_t pos, hi;
    int b;
    bool fresh;
};

__device__ __forceinline__ int tiles_of(uint32_t act) { return static_cast<int>((act + kBS - 1) / kBS); }

// weight of one kv head of a sequence with `rows` query rows a kv head
__device__ __forceinline__ uint32_t head_weight(uint32_t rows, uint32_t tiles)
{
    if (rows == 0 || tiles == 0) return 0;
    return (rows + kItemRows - 1) / kItemRows * (tiles + kItemCost);
}

// the item at `pos` of sequence s.b, whose first position is base0; its first
// position and the one behind it
__device__ __forceinline__ void locate(uint32_t pos, uint32_t base0, int rows_b, int tiles, Seg& s, uint32_t& base,
                                       uint32_t& end)
{
    const uint32_t per_head = head_weight(rows_b, tiles);
    const uint32_t rem = pos - base0;
    s.h = static_cast<int>(rem / per_head);
    const uint32_t full = tiles + kItemCost;
    const int item = static_cast<int>((rem - s.h * per_head) / full);
    s.row0 = item * kItemRows;
    s.rows = min(rows_b - s.row0, kItemRows);
    s.tiles = tiles;
    base = base0 + s.h * per_head + item * full;
    end = base + full;
}

// blocks of item `s` before position `off` behind its first one
__device__ __forceinline__ int blocks_before(const Seg& s, uint32_t off)
{
    return min(static_cast<int>(off > kItemCost ? off - kItemCost : 0u), s.tiles);
}

// The run's next item with blocks [t0, t1) in it.
__device__ __forceinline__ bool next_seg(const uint32_t* cum, const uint32_t* len, int G, Run& r, Seg& s)
{
    while (r.pos < r.hi) {
        while (cum[r.b + 1] <= r.pos) ++r.b;
        s.b = r.b;
        uint32_t base, end;
        locate(r.pos, cum[r.b], static_cast<int>(len[r.b] & 0xFF) * G, tiles_of(len[r.b] >> 8), s, base, end);
        s.t0 = blocks_before(s, r.pos - base);
        s.t1 = r.hi >= end ? s.tiles : blocks_before(s, r.hi - base);
        s.first = r.fresh;
        r.fresh = false;
        r.pos = min(end, r.hi);
        if (s.t0 < s.t1) return true;
    }
    return false;
}

// The drafted token of a query row of a kv head (exact: the row is below 2^14,
// the factor's error times it below 1 / 128).
__device__ __forceinline__ int node_of(const TreeParams& p, int row)
{
    return static_cast<int>((static_cast<uint64_t>(row) * p.g_mul) >> 22);
}

// Row r of item `s` in q and out.
__device__ __forceinline__ int q_row(const TreeParams& p, const Seg& s, int r)
{
    const int rr = s.row0 + r, node = node_of(p, rr);
    return (s.b * p.S1 + node) * p.NQ + s.h * p.G + (rr - node * p.G);
}

__device__ __forceinline__ float* part_of(const TreeParams& p, int cta, bool first)
{
    return p.part + (static_cast<int64_t>(cta) * 2 + (first ? 0 : 1)) * p.part_rows * (kD + 2);
}

// ---- the warps' parts ------------------------------------------------------------------
__device__ void producer(TreeSmem& sm, const TreeParams& p, const CUtensorMap* tk, const CUtensorMap* tv, Run run,
                         int lane)
{
    const uint64_t pol = p.keep_l2 ? l2_keep_policy() : l2_evict_first_policy();
    Seg s;
    int kc = 0, vc = 0;                      // blocks requested so far
    bool stop = false;
    while (!stop && next_seg(sm.cum, sm.len, p.G, run, s)) {
        const int* row = p.bt + static_cast<int64_t>(s.b) * p.max_blocks;
        int ids = 0;
        for (int t = s.t0; t < s.t1; ++t) {
            const int at = (t - s.t0) & 31;
            if (at == 0) {
                ids = t + lane < s.t1 ? __ldg(row + t + lane) : 0;
                if (ids < 0 || ids >= p.num_blocks) ids = 0;
            }
            const int64_t blk = __shfl_sync(0xffffffffu, ids, at);
            const int x = p.layout == PA_LAYOUT_BSND ? s.h * kD : 0;
            const int y = static_cast<int>(p.layout == PA_LAYOUT_BSND ? blk * kBS : (blk * p.NKV + s.h) * kBS);
            const int kslot = kc % kKStages, vslot = vc % kVStages, sslot = kc % kSStages;
            if (!wait_for(&sm.k_empty[kslot], ((kc / kKStages) & 1) ^ 1, p.err, 1, &sm.abort)) stop = true;
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
            if (!wait_for(&sm.v_empty[vslot], ((vc / kVStages) & 1) ^ 1, p.err, 2, &sm.abort)) stop = true;
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

// V codes [key][channel] (128-byte swizzled rows) to FP16 in two chunks of 64
// channels, swizzled the same way; keys at and behind `act` become zeros, so
// that no stale code (a NaN among them) meets their P = 0.
__device__ void converter(TreeSmem& sm, const TreeParams& p, Run run, int w, int lane)
{
    // Lane l takes 16-byte unit u = l % 8 of eight rows whose numbers differ in
    // the 8-row group only, so that every address is a constant away from the
    // first. Units 4-7 go with the neighbouring row: a unit becomes two of one
    // chunk, and units u and u + 4 of a row would meet in the banks.
    Seg s;
    int c = 0;
    const int u = lane & 7;
    const int key0 = 64 * (w >> 1) + 4 * (w & 1) + ((lane >> 3) ^ (u >> 2));
    const uint32_t from = sw128(key0, u), to = sw128(key0, 2 * (u & 3)) + (u >> 2) * kTile,
                   to1 = sw128(key0, 2 * (u & 3) + 1) + (u >> 2) * kTile;
    while (next_seg(sm.cum, sm.len, p.G, run, s)) {
        const int act = static_cast<int>(sm.len[s.b] >> 8);
        for (int t = s.t0; t < s.t1; ++t, ++c) {
            const int vslot = c % kVStages, hslot = c % kHStages;
            wait_for(&sm.v_full[vslot], (c / kVStages) & 1, p.err, 4, &sm.abort);
            const uint8_t* src = sm.v[vslot] + from;
            const int limit = act - t * kBS;
            wait_for(&sm.h_empty[hslot], ((c / kHStages) & 1) ^ 1, p.err, 8, &sm.abort);
            uint8_t* dst = sm.vh[hslot][0];
#pragma unroll
            for (int i0 = 0; i0 < 8; i0 += 4) {
                uint4 x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint4*>(src + 1024 * (i0 + i));
                if (limit < kBS) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (key0 + 8 * (i0 + i) >= limit) x[i] = make_uint4(0, 0, 0, 0);
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
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.h_full[hslot]);
                mbar_arrive(&sm.v_empty[vslot]);
            }
        }
    }
}

// The MMAs' two warps: the whole warp waits, one elected thread issues. Warp 0
// issues S, as far ahead as there are K blocks and free S buffers, warp 1 P V.
__device__ void mma_issuer(TreeSmem& sm, const TreeParams& p, Run run, uint32_t tmem, int w)
{
    constexpr uint32_t kIdescS = idesc_e4m3(128, kBS, 0, 0);
    constexpr uint32_t kIdescO = idesc_f16(128, kD, 0, 1);   // P K-major in tensor memory, V MN-major
    auto wait = [&](uint64_t* bar, int phase, int code) {
        return __all_sync(0xffffffffu, wait_for(bar, phase & 1, p.err, code, &sm.abort)) != 0;
    };
    Seg s;
    int i = 0, seg = 0;                      // blocks, segments so far
    bool ok = true;
    while (ok && next_seg(sm.cum, sm.len, p.G, run, s)) {
        if (w == 0) ok = wait(&sm.q_full[seg & 1], seg >> 1, 16);
        const uint64_t qd = smem_desc(smem_u32(sm.q[seg & 1]), 16, 1024, kSmem128BSwizzle);
#pragma unroll 1
        for (int t = s.t0; t < s.t1 && ok; ++t, ++i) {
            const int buf = i % kTurns, turn = i / kTurns, kslot = i % kKStages, hslot = i % kHStages;
            if (w == 0)
                ok = wait(&sm.k_full[i % kSStages], i / kSStages, 16) &&
                     (turn == 0 || wait(&sm.s_free[buf], turn - 1, 32));
            else
                ok = wait(&sm.h_full[hslot], i / kHStages, 32) && wait(&sm.p_full[buf], turn, 32);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                if (w == 0) {
                    const uint64_t kd = smem_desc(smem_u32(sm.k[kslot]), 16, 1024, kSmem128BSwizzle);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_e4m3(tmem + kSCol + kBS * buf, qd + 2 * kk, kd + 2 * kk, kIdescS, kk);
                    umma_commit(&sm.s_full[buf]);
                    umma_commit(&sm.k_empty[kslot]);
                    if (t + 1 == s.t1) umma_commit(&sm.q_empty[seg & 1]);
                } else {
                    const uint64_t vd = smem_desc(smem_u32(sm.vh[hslot][0]), kTile, 1024, kSmem128BSwizzle);
#pragma unroll
                    for (int kk = 0; kk < kBS / 16; ++kk)   // 16 keys: 8 columns of P, 2048 bytes of V
                        umma_f16_ta(tmem, tmem + kPCol + kBS / 2 * buf + 8 * kk, vd + 128 * kk, kIdescO,
                                    (t > s.t0 || kk > 0) ? 1u : 0u);
                    umma_commit(&sm.o_done[buf]);
                    umma_commit(&sm.h_empty[hslot]);
                }
            }
            __syncwarp();
        }
        ++seg;
    }
    if (elect_one()) {
        umma_commit(&sm.drain[w]);
        mbar_wait_drain(&sm.drain[w], 0, p.err, 512);
    }
    __syncwarp();
}

// Q rows (128-byte swizzled), q_scale and v_scale of each segment, ahead of the
// softmax by one.
__device__ void q_loader(TreeSmem& sm, const TreeParams& p, Run run, int lane)
{
    Seg s;
    for (int seg = 0; next_seg(sm.cum, sm.len, p.G, run, s); ++seg) {
        const int buf = seg & 1;
        if (!__all_sync(0xffffffffu, wait_for(&sm.q_empty[buf], ((seg >> 1) & 1) ^ 1, p.err, 1024, &sm.abort))) break;
#pragma unroll 4
        for (int i = 0; i < 32; ++i) {
            const int r = 4 * i + (lane >> 3), u = lane & 7;
            const bool in = r < s.rows;
            const int64_t at = q_row(p, s, in ? r : 0);
            cp_async16(sm.q[buf] + sw128(r, u), p.q + at * kD + 16 * u, in ? 16 : 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 32 * i + lane;
            cp_async4(&sm.qs[buf][r], p.q_scale + q_row(p, s, r < s.rows ? r : 0), 4);
        }
        cp_async16(&sm.vs[buf][4 * lane], p.v_scale + static_cast<int64_t>(s.b * p.NKV + s.h) * kD + 4 * lane, 16);
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_full[buf]);
    }
}

// Warpgroup w: blocks w, w + kTurns, ..; the thread of row `row`.
__device__ void softmax(TreeSmem& sm, const TreeParams& p, Run run, uint32_t tmem, int w, int q4, int lane)
{
    const int row = 32 * q4 + lane;
    // named barriers: a warp decides on m for its block, the next warpgroup's warp of
    // the same rows waits for that
    const int mine = 2 + kTurns * q4 + w, theirs = 2 + kTurns * q4 + (w + kTurns - 1) % kTurns;
    const uint32_t O = tmem + (static_cast<uint32_t>(32 * q4) << 16);
    const uint32_t S = O + kSCol + kBS * w, P = O + kPCol + kBS / 2 * w;
    // The next segment, and the row's mask in it, one bit per drafted token: a ballot
    // per node of the warp's rows and 32 drafted tokens, eight of them loaded at once.
    Seg s;
    uint64_t m_lo = 0, m_hi = 0;
    auto advance = [&] {
        if (!next_seg(sm.cum, sm.len, p.G, run, s)) return false;
        const int act = static_cast<int>(sm.len[s.b] >> 8), n = static_cast<int>(sm.len[s.b] & 0xFF);
        m_lo = m_hi = 0;
        if (32 * q4 >= s.rows || s.t1 * kBS <= act - n) return true;
        const int first = node_of(p, s.row0 + 32 * q4), own = node_of(p, s.row0 + row);
        const int last = node_of(p, s.row0 + min(32 * q4 + 31, s.rows - 1));
        const uint8_t* mr = p.mask + s.b * p.mask_stride + static_cast<int64_t>(first) * p.S1;
        int node = first, j = 0;
#pragma unroll 1
        while (node <= last) {
            int nodes[8], js[8];
            bool see[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                nodes[i] = node;
                js[i] = j;
                see[i] = node <= last && j + lane < n && __ldg(mr + j + lane);
                j += 32;
                if (j >= n) {
                    j = 0;
                    ++node;
                    mr += p.S1;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t bits = __ballot_sync(0xffffffffu, see[i]);
                if (nodes[i] == own) (js[i] < 64 ? m_lo : m_hi) |= static_cast<uint64_t>(bits) << (js[i] & 32);
            }
        }
        return true;
    };
    int g0 = 0, turn = 0, next = w;          // blocks in all so far, own ones, the next own one
    bool more = advance();
#pragma unroll 1
    for (int seg = 0; more; ++seg) {
        const int ctx = static_cast<int>(sm.len[s.b] >> 8) - static_cast<int>(sm.len[s.b] & 0xFF);
        const bool warp_live = 32 * q4 < s.rows, live = row < s.rows;
        wait_for(&sm.q_full[seg & 1], (seg >> 1) & 1, p.err, 64, &sm.abort);
        float rs = live ? sm.qs[seg & 1][row] * p.scale_log2 : 1.0f;
        // the maximum of S k_scale has to stay one under a negative scale: S changes sign
        const bool flip = rs < 0.0f, any_flip = __any_sync(0xffffffffu, flip);
        rs = fabsf(rs);
        if (rs < 1.17549435e-38f) rs = 1.17549435e-38f;       // (-inf times it stays -inf; a NaN stays, too)
        float m = -INFINITY, l = 0.0f;
        const int g_end = g0 + (s.t1 - s.t0);
        // A warp without rows keeps the others company at the barriers.
        for (; next < g_end && !warp_live; next += kTurns, ++turn) {
            wait_for(&sm.s_full[w], turn & 1, p.err, 64, &sm.abort);
            if (lane == 0) mbar_arrive(&sm.s_free[w]);
            if (turn > 0) wait_for(&sm.o_done[w], (turn - 1) & 1, p.err, 128, &sm.abort);
            if (lane == 0) mbar_arrive(&sm.p_full[w]);
        }
#pragma unroll 1
        for (; next < g_end && warp_live; next += kTurns, ++turn) {
            const int slot = next % kSStages;
            wait_for(&sm.s_full[w], turn & 1, p.err, 64, &sm.abort);
            tc_fence_after();
            wait_for(&sm.k_full[slot], (next / kSStages) & 1, p.err, 64, &sm.abort);
            __syncwarp();
            float v[kBS];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(S + 32 * c, v + 32 * c);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.s_free[w]);
            const float4* ks = reinterpret_cast<const float4*>(sm.ks[slot]);
#pragma unroll
            for (int c = 0; c < kBS / 4; ++c) {
                const float4 k4 = ks[c];
                const float2 a = __fmul2_rn(make_float2(v[4 * c], v[4 * c + 1]), make_float2(k4.x, k4.y));
                const float2 b = __fmul2_rn(make_float2(v[4 * c + 2], v[4 * c + 3]), make_float2(k4.z, k4.w));
                v[4 * c] = a.x;
                v[4 * c + 1] = a.y;
                v[4 * c + 2] = b.x;
                v[4 * c + 3] = b.y;
            }
            if (any_flip) {
#pragma unroll
                for (int k = 0; k < kBS; ++k) v[k] = flip ? -v[k] : v[k];
            }
            const int off = ctx - (s.t0 + next - g0) * kBS;     // the first drafted token's key here
            if (off < kBS) {
                // which keys the row sees: the context's, then its mask's bits
                uint64_t lo, hi;
                if (off >= 64) {
                    lo = ~0ull;
                    hi = (off == 64 ? 0ull : ~0ull >> (128 - off)) | (m_lo << (off - 64));
                } else if (off > 0) {
                    lo = (~0ull >> (64 - off)) | (m_lo << off);
                    hi = (m_hi << off) | (m_lo >> (64 - off));
                } else if (off == 0) {
                    lo = m_lo;
                    hi = m_hi;
                } else if (off > -64) {
                    lo = (m_lo >> -off) | (m_hi << (64 + off));
                    hi = m_hi >> -off;
                } else {
                    lo = off > -128 ? m_hi >> (-off - 64) : 0ull;
                    hi = 0ull;
                }
#pragma unroll
                for (int k = 0; k < 64; ++k) {
                    if (!((lo >> k) & 1)) v[k] = -INFINITY;
                    if (!((hi >> k) & 1)) v[64 + k] = -INFINITY;
                }
            }
            float m4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                m4[c] = fmaxf(v[32 * c], v[32 * c + 1]);
#pragma unroll
                for (int k = 2; k < 32; k += 2) m4[c] = max3(m4[c], v[32 * c + k], v[32 * c + k + 1]);
            }
            const float mx = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]) * rs;
            // Past 2^22 the rounding of mx is no longer small beside the exponents, which
            // take the products unrounded (one too large by 1 leaves FP16): there they are
            // rounded as mx is. (Rounding all of them takes 2 to 3% longer.)
            const bool big = fabsf(mx) > 0x1p22f;
            float rx = rs;
            if (__builtin_expect(__any_sync(0xffffffffu, big), 0)) {
                const float f = big ? rs : 1.0f;
#pragma unroll
                for (int k = 0; k < kBS; ++k) v[k] *= f;
                rx = big ? 1.0f : rs;
            }
            // this P buffer's last P V is complete
            if (turn > 0) wait_for(&sm.o_done[w], (turn - 1) & 1, p.err, 128, &sm.abort);
            __syncwarp();
            // ---- m, after the block before ----
            const bool later = next > g0;                      // a block of the segment lies before this one
            float mn = -INFINITY;
            if (later) {
                named_bar_sync(theirs, 64);
                mn = sm.m[row];
            }
            const bool raise = mx > mn + kRaise || (mn == -INFINITY && mx > -INFINITY);
            if (__any_sync(0xffffffffu, raise)) {
                const float old = mn;
                mn = raise ? mx : mn;
                if (later) {
                    // O is complete before it is scaled (and its barrier's phase is the
                    // one waited for: the other warp waited for that before its decision)
                    wait_for(&sm.o_done[(next - 1) % kTurns], ((next - 1) / kTurns) & 1, p.err, 128, &sm.abort);
                    __syncwarp();
                    tc_fence_after();
                    const float f = raise ? ex2(old - mn) : 1.0f;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        float o[32];
                        tmem_ld32(O + 32 * c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] *= f;
                        tmem_st32(O + 32 * c, o);
                    }
                    tmem_wait_st();
                }
            }
            sm.m[row] = mn;
            if (next + 1 < g_end) named_bar_arrive(mine, 64);
            l *= mn != m ? ex2(m - mn) : 1.0f;                 // (0 while m is -inf)
            m = mn;
            tc_fence_after();
            const float ref = m == -INFINITY ? 0.0f : m - kShift;
            const float2 rs2 = make_float2(rx, rx), nref = make_float2(-ref, -ref);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t hp[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float2 x = __ffma2_rn(make_float2(v[32 * c + 2 * k], v[32 * c + 2 * k + 1]), rs2, nref);
                    x.x = ex2(x.x);
                    x.y = ex2(x.y);
                    sum[k & 1] = __fadd2_rn(sum[k & 1], x);
                    hp[k] = half2_bits(x.x, x.y);
                }
                tmem_st16(P + 16 * c, hp);
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full[w]);
        }
        g0 = g_end;
        // ---- the item's (or its part's) output, 32 channels at a time in turn ----
        sm.ml[0][w][row] = m;
        sm.ml[1][w][row] = l;
        __syncwarp();
        named_bar_sync(1, 4 * kTurns * 32);
        // (the next segment's, while the last P V goes on)
        const Seg done = s;
        more = advance();
        // the last P V, and with it all (one accumulator: they complete in order);
        // behind the barrier, as its warpgroup waited for this barrier's last phase
        wait_for(&sm.o_done[(g_end - 1) % kTurns], ((g_end - 1) / kTurns) & 1, p.err, 128, &sm.abort);
        __syncwarp();
        tc_fence_after();
        if (warp_live) {
            const float mf = sm.m[row];      // the last decision's
            float lt = 0.0f;
#pragma unroll
            for (int k = 0; k < kTurns; ++k) {
                const float mk = sm.ml[0][k][row];
                lt += sm.ml[1][k][row] * (mk == mf ? 1.0f : ex2(mk - mf));
            }
            const bool whole = done.t0 == 0 && done.t1 == done.tiles;
            const float inv = lt == 0.0f ? 0.0f : __fdiv_rn(1.0f, lt);
            const int at = live ? q_row(p, done, row) : -1;
            float* const part = part_of(p, blockIdx.x, done.first);
#pragma unroll 1
            for (int c = w; c < kD / 32; c += kTurns) {
                __syncwarp();                // (rows behind the last one store nothing)
                float o[32];
                tmem_ld32(O + 32 * c, o);
                tmem_wait_ld();
                if (!live) continue;
                if (whole) {
                    const float4* vs = reinterpret_cast<const float4*>(sm.vs[seg & 1] + 32 * c);
                    uint4* dst = reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(at) * kD + 32 * c);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 a = vs[2 * k], e = vs[2 * k + 1];
                        const float* x = o + 8 * k;
                        const __nv_bfloat162 y0 = __floats2bfloat162_rn(x[0] * inv * a.x, x[1] * inv * a.y);
                        const __nv_bfloat162 y1 = __floats2bfloat162_rn(x[2] * inv * a.z, x[3] * inv * a.w);
                        const __nv_bfloat162 y2 = __floats2bfloat162_rn(x[4] * inv * e.x, x[5] * inv * e.y);
                        const __nv_bfloat162 y3 = __floats2bfloat162_rn(x[6] * inv * e.z, x[7] * inv * e.w);
                        dst[k] = make_uint4(
                            *reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1),
                            *reinterpret_cast<const uint32_t*>(&y2), *reinterpret_cast<const uint32_t*>(&y3));
                    }
                } else {
                    float4* dst = reinterpret_cast<float4*>(part + row * kD + 32 * c);
#pragma unroll
                    for (int k = 0; k < 8; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                }
            }
            if (!whole && live && w == 0) {
                float* ml = part + static_cast<int64_t>(p.part_rows) * kD;
                ml[row] = mf;
                ml[p.part_rows + row] = lt;
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_empty[seg & 1]);
        __syncwarp();
        // (O, m and l of this segment are not touched before all are here)
        named_bar_sync(1, 4 * kTurns * 32);
    }
}

// What the joining kernel has to know of the item at the begin of this CTA's run.
// Runs c0 to c1, those with its first and its last block's positions, have a block
// of it each (a position behind the first block's is a block's), and no other run
// has one. Empty runs lie behind the last item.
__device__ void describe_cut(TreeSmem& sm, const TreeParams& p, const Run& run, uint32_t total, int lane)
{
    const int c = blockIdx.x;
    Cut cut = {};
    if (run.pos < total && c > 0) {
        Seg s;
        s.b = run.b;                         // (holds run.pos: the run is not empty)
        uint32_t base, end;
        locate(run.pos, sm.cum[s.b], static_cast<int>(sm.len[s.b] & 0xFF) * p.G, tiles_of(sm.len[s.b] >> 8), s, base,
               end);
        if (run.pos > base) {
            const int c0 = cta_of(total, base + kItemCost, p.ctas), c1 = cta_of(total, end - 1, p.ctas);
            if (c == c0 + 1 && c0 < c1) {
                cut.b = s.b;
                cut.h = s.h;
                cut.row0 = s.row0;
                cut.rows = s.rows;
                cut.c0 = c0;
                cut.c1 = c1;
                cut.slot0 = 2 * c0 + (run_begin(total, c0, p.ctas) >= base ? 0 : 1);
            }
        }
    }
    if (lane == 0) p.cuts[c] = cut;
}

__global__ void __launch_bounds__(kThreads, 1)
    tree_decode_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const TreeParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uintptr_t raw = reinterpret_cast<uintptr_t>(smem_raw);
    TreeSmem& sm = *reinterpret_cast<TreeSmem*>(smem_raw + ((1024u - (raw & 1023u)) & 1023u));
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
        for (int i = 0; i < kTurns; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_free[i], 4);
            mbar_init(&sm.p_full[i], 4);
            mbar_init(&sm.o_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.q_empty[i], 1 + 4 * kTurns);
            mbar_init(&sm.drain[i], 1);
        }
        sm.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(&sm.tmem, kTmemCols);
    grid_launch_dependents();   // (the joining kernel waits for this one's end)

    // ---- weights before each sequence: thread i takes sequences i, i + 1, ... of its share ----
    {
        const int per = (p.B + kThreads - 1) / kThreads;
        uint32_t mine = 0;
        for (int b = tid * per; b < min(p.B, tid * per + per); ++b) {
            const int act = min(max(__ldg(p.act + b), 0), p.max_blocks * kBS);
            int n = p.len ? __ldg(p.len + b) : p.S1;
            n = min(max(n, 0), min(p.S1, act));
            sm.len[b] = static_cast<uint32_t>(act) << 8 | static_cast<uint32_t>(n);
            sm.cum[b] = mine;
            mine += p.NKV * head_weight(n * p.G, tiles_of(act));
        }
        uint32_t x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        uint32_t* const warp_sum = reinterpret_cast<uint32_t*>(sm.ml);
        if (lane == 31) warp_sum[warp] = x;
        __syncthreads();
        uint32_t before = x - mine;
        for (int i = 0; i < warp; ++i) before += warp_sum[i];
        for (int b = tid * per; b < min(p.B, tid * per + per); ++b) sm.cum[b] += before;
        if (tid == kThreads - 1) sm.cum[p.B] = before + mine;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const uint32_t total = sm.cum[p.B];
    Run run;
    run.pos = run_begin(total, blockIdx.x, p.ctas);
    run.hi = run_begin(total, blockIdx.x + 1, p.ctas);
    run.fresh = true;
    run.b = 0;
    if (run.pos < run.hi) {
        int lo = 0, hi = p.B - 1;            // the last sequence that starts at or before pos
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (sm.cum[mid] <= run.pos) lo = mid;
            else hi = mid - 1;
        }
        run.b = lo;
    }

    if (warp < kProdWarp) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        softmax(sm, p, run, tmem, warp >> 2, warp & 3, lane);
    } else if (warp < kConvWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kProdWarp) {
            producer(sm, p, &tk, &tv, run, lane);
            // (behind the Q loader instead 16 x 64 drafted tokens take 150 us, not 129)
            describe_cut(sm, p, run, total, lane);
        } else if (warp == kQWarp) {
            q_loader(sm, p, run, lane);
        } else {
            mma_issuer(sm, p, run, tmem, warp - kMmaWarp);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        // rows that see nothing because their sequence has no such node
        for (int64_t tok = blockIdx.x; tok < static_cast<int64_t>(p.B) * p.S1; tok += gridDim.x) {
            const int b = static_cast<int>(tok / p.S1);
            if (tok - static_cast<int64_t>(b) * p.S1 < (sm.len[b] & 0xFF)) continue;
            uint4* dst = reinterpret_cast<uint4*>(p.out + tok * p.NQ * kD);
            for (int i = tid - kConvWarp * 32; i < p.NQ * (kD / 8); i += kConvWarps * 32) dst[i] = make_uint4(0, 0, 0, 0);
        }
        converter(sm, p, run, warp - kConvWarp, lane);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the parts of the items that a run's end cut: CTA (c, y) takes the item
// whose first block run c has and whose last one a later run, a warp two rows of it
// and four parts at once, all their loads in flight together. Launched early, it
// still adds 4 to 5 us to a call: the decode's CTAs leave no room beside them, so
// it starts when they end, and its loads are a chain of two (the cut, then parts).
// (Factors from all maxima first, a third link, took 1.5 us more on 131072 keys;
// joining in the decode's own last CTAs lost more in the decode than this costs.)
constexpr int kJoinWarps = 4, kJoinRows = 2, kJoinParts = 4;

__global__ void __launch_bounds__(kJoinWarps * 32) tree_join_kernel(const TreeParams p)
{
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int4 a = *reinterpret_cast<const int4*>(p.cuts + blockIdx.x + 1);
    const int4 z = *(reinterpret_cast<const int4*>(p.cuts + blockIdx.x + 1) + 1);
    Seg s;
    s.b = a.x;
    s.h = a.y;
    s.row0 = a.z;
    s.rows = a.w;
    const int row0 = (blockIdx.y * kJoinWarps + (threadIdx.x >> 5)) * kJoinRows;
    if (row0 >= s.rows) return;
    const int c0 = z.x, c1 = z.y, slot0 = z.z;
    const int64_t slot_floats = static_cast<int64_t>(p.part_rows) * (kD + 2);
    // O's part of run c (its rows begin there), m and l behind the rows; rows
    // past the item's last are read from it and not written
    auto part = [&](int c) { return p.part + (c == c0 ? slot0 : 2 * c) * slot_floats; };
    const float4 v =
        __ldg(reinterpret_cast<const float4*>(p.v_scale + static_cast<int64_t>(s.b * p.NKV + s.h) * kD) + lane);
    int row[kJoinRows];
    float M[kJoinRows], L[kJoinRows];
    float4 o[kJoinRows];
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) {
        row[r] = min(row0 + r, s.rows - 1);
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
                // nothing seen in this part. (Where all scores are NaN the maximum is -inf
                // as well, and the sum NaN: that has to reach the output.)
                if (l[i][r] == 0.0f) continue;
                const float mn = fmaxf(M[r], m[i][r]), f = ex2(M[r] - mn), g = ex2(m[i][r] - mn);
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
        if (row0 + r >= s.rows) break;
        const float inv = L[r] == 0.0f ? 0.0f : __fdiv_rn(1.0f, L[r]);
        const __nv_bfloat162 y0 = __floats2bfloat162_rn(o[r].x * inv * v.x, o[r].y * inv * v.y);
        const __nv_bfloat162 y1 = __floats2bfloat162_rn(o[r].z * inv * v.z, o[r].w * inv * v.w);
        reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(q_row(p, s, row[r])) * kD)[lane] =
            make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
    }
}

// rows of the largest item, a multiple of 64 so that parts start on 256 bytes
int part_rows(int S1, int G)
{
    const int64_t r = static_cast<int64_t>(S1) * G;
    return r >= kItemRows ? kItemRows : static_cast<int>((r + 63) / 64 * 64);
}

pa_status check_shape(const char* name, int B, int S1, int NQ, int NKV, int D)
{
    PA_REQUIRE(B >= 0 && S1 > 0 && NQ > 0 && NKV > 0 && D > 0, PA_ERR_INVALID,
               "%s: negative or empty shape (B=%d S1=%d NQ=%d NKV=%d D=%d)", name, B, S1, NQ, NKV, D);
    PA_REQUIRE(NQ % NKV == 0, PA_ERR_INVALID, "%s: NQ %d is not a multiple of NKV %d", name, NQ, NKV);
    PA_REQUIRE(D == kD, PA_ERR_UNSUPPORTED, "%s: head size %d (only 128 is built)", name, D);
    PA_REQUIRE(B <= kMaxB, PA_ERR_UNSUPPORTED, "%s: batch %d > %d", name, B, kMaxB);
    PA_REQUIRE(S1 <= kMaxNodes, PA_ERR_UNSUPPORTED, "%s: S1 %d > %d drafted tokens", name, S1, kMaxNodes);
    PA_REQUIRE(NQ / NKV <= kMaxGroup, PA_ERR_UNSUPPORTED, "%s: %d query heads per kv head (at most %d)", name,
               NQ / NKV, kMaxGroup);
    return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_fp8_tree_decode_workspace_size(int B, int S1, int NQ, int NKV, int D, size_t* bytes)
{
    PA_REQUIRE(bytes, PA_ERR_NULLPTR, "pa_fp8_tree_decode_workspace_size: bytes is NULL");
    const pa_status st = check_shape("pa_fp8_tree_decode", B, S1, NQ, NKV, D);
    if (st != PA_OK) return st;
    *bytes = kPartOff + static_cast<size_t>(kMaxCtas) * 2 * part_rows(S1, NQ / NKV) * (kD + 2) * sizeof(float);
    return PA_OK;
}

extern "C" pa_status pa_fp8_tree_decode(const void* q, const float* q_scale, const void* k_cache,
                                        const float* k_scale, const void* v_cache, const float* v_scale,
                                        const int32_t* block_table, const int32_t* kv_act_seqs,
                                        const int32_t* tree_len, const uint8_t* tree_mask, int64_t mask_stride,
                                        void* out, int B, int S1, int NQ, int NKV, int D, int block_size,
                                        int64_t num_blocks, int max_blocks_per_seq, int layout,
                                        float softmax_scale, void* workspace, size_t workspace_bytes,
                                        void* stream)
{
    const char* name = "pa_fp8_tree_decode";
    // (tensors of no sequences may have no address)
    PA_REQUIRE(k_cache && k_scale && v_cache &&
                   (B == 0 || (q && q_scale && v_scale && block_table && kv_act_seqs && tree_mask && out)),
               PA_ERR_NULLPTR, "%s: NULL tensor pointer", name);
    size_t need = 0;
    const pa_status ps = pa_fp8_tree_decode_workspace_size(B, S1, NQ, NKV, D, &need);
    if (ps != PA_OK) return ps;
    PA_REQUIRE(num_blocks > 0 && max_blocks_per_seq > 0 && block_size > 0, PA_ERR_INVALID,
               "%s: empty cache or block table", name);
    PA_REQUIRE(block_size == kBS, PA_ERR_UNSUPPORTED, "%s: block_size %d (only 128 is built)", name, block_size);
    PA_REQUIRE(layout == PA_LAYOUT_BSND || layout == PA_LAYOUT_BNBD, PA_ERR_INVALID, "%s: unknown layout %d", name,
               layout);
    PA_REQUIRE(max_blocks_per_seq < (1 << 24) / kBS, PA_ERR_UNSUPPORTED,
               "%s: block table of %d blocks, 2^24 positions or more", name, max_blocks_per_seq);
    PA_REQUIRE(num_blocks * kBS * NKV <= 0x7FFFFFFF, PA_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 cache rows", name);
    PA_REQUIRE(std::isfinite(softmax_scale), PA_ERR_INVALID, "%s: softmax_scale not finite", name);
    PA_REQUIRE(mask_stride >= 0, PA_ERR_INVALID, "%s: negative mask_stride", name);
    PA_REQUIRE(aligned16(q) && aligned16(k_cache) && aligned16(v_cache) && aligned16(v_scale) && aligned16(out),
               PA_ERR_INVALID, "%s: q, the caches, v_scale and out must be 16-byte aligned", name);
    for (const void* x : {static_cast<const void*>(q_scale), static_cast<const void*>(k_scale),
                          static_cast<const void*>(block_table), static_cast<const void*>(kv_act_seqs),
                          static_cast<const void*>(tree_len)})
        PA_REQUIRE((reinterpret_cast<uintptr_t>(x) & 3u) == 0, PA_ERR_INVALID,
                   "%s: q_scale, k_scale, block_table, kv_act_seqs and tree_len must be 4-byte aligned", name);
    // the schedule counts blocks in 32 bits
    const int64_t per_block = (static_cast<int64_t>(S1) * (NQ / NKV) + kItemRows - 1) / kItemRows * (1 + kItemCost);
    PA_REQUIRE(per_block * NKV * B <= 0xFFFFFFFFll / max_blocks_per_seq, PA_ERR_UNSUPPORTED,
               "%s: B * heads * max_blocks_per_seq too large for the 32-bit schedule", name);
    PA_REQUIRE(static_cast<int64_t>(B) * S1 * NQ <= 0x7FFFFFFF, PA_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 query rows",
               name);
    if (B == 0) return PA_OK;
    PA_REQUIRE(workspace && workspace_bytes >= need, PA_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", name,
               workspace ? workspace_bytes : static_cast<size_t>(0), need);
    PA_REQUIRE((reinterpret_cast<uintptr_t>(workspace) & 255u) == 0, PA_ERR_INVALID,
               "%s: workspace must be 256-byte aligned", name);
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
    TreeParams p;
    p.q = static_cast<const uint8_t*>(q);
    p.q_scale = q_scale;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.bt = block_table;
    p.act = kv_act_seqs;
    p.len = tree_len;
    p.mask = tree_mask;
    p.mask_stride = mask_stride;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.err = reinterpret_cast<int*>(ws);
    p.cuts = reinterpret_cast<Cut*>(ws + kCutOff);
    p.part = reinterpret_cast<float*>(ws + kPartOff);
    p.part_rows = part_rows(S1, NQ / NKV);
    p.B = B;
    p.S1 = S1;
    p.NQ = NQ;
    p.NKV = NKV;
    p.G = NQ / NKV;
    p.g_mul = (1u << 22) / p.G + 1;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    p.layout = layout;
    p.ctas = sms < kMaxCtas ? sms : kMaxCtas;
    p.keep_l2 = static_cast<int64_t>(S1) * p.G > kItemRows;
    p.scale_log2 = softmax_scale * 1.4426950408889634f;

    cudaError_t e = cudaFuncSetAttribute(tree_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSmemBytes));
    PA_REQUIRE(e == cudaSuccess, PA_ERR_CUDA, "%s: smem attribute: %s", name, cudaGetErrorString(e));
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    tree_decode_kernel<<<static_cast<unsigned>(p.ctas), kThreads, kSmemBytes, cs>>>(tk, tv, p);
    st = check_launch(name);
    if (st != PA_OK || p.ctas == 1) return st;
    const int64_t most = static_cast<int64_t>(S1) * p.G < kItemRows ? static_cast<int64_t>(S1) * p.G : kItemRows;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(p.ctas - 1), static_cast<unsigned>((most + kJoinWarps * kJoinRows - 1) / (kJoinWarps * kJoinRows)));
    lc.blockDim = dim3(kJoinWarps * 32);
    lc.stream = cs;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    e = cudaLaunchKernelEx(&lc, tree_join_kernel, p);
    PA_REQUIRE(e == cudaSuccess, PA_ERR_CUDA, "%s: launch: %s", name, cudaGetErrorString(e));
    return PA_OK;
}
