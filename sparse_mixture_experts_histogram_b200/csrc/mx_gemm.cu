// mx_gemm.cu -- products of microscaled rows with 4-bit expert weights, on
// CTA pairs with block-scaled tensor-core MMAs (tcgen05 .cta_group::2
// .block_scale):
//   y[r, n] = sum_k W_e[n, k] x[r, k]                   (moe_mx_product)
//   h[r, f] = act(W1_e x[r])[f] * (W3_e x[r])[f]        (moe_mx_gated)
// for every row r of expert e's segment, cut into token tiles of near-equal
// size.  W is e2m1, x e4m3 (kind::mxf8f6f4) or e2m1 (kind::mxf4, twice the
// rate), one power-of-two scale per 32 values of K on both sides; the tensor
// cores multiply the scales in and sum in fp32.
//
// The weights are the MMA's A operand (M = 256 over the pair), a tile's rows
// its B operand (N = rows rounded up to 16, half of them in each CTA): a
// ragged segment costs the MMA columns it needs, and the same kernel streams
// the weights for a single token.  Each CTA holds 128 weight rows: of the
// product 128 output columns, of the gated form 64 rows of W1 and the same 64
// of W3, so that both sums of an output lie in one CTA.
//
// Operands reach shared memory as 128-byte rows by TMA, two columns of 128
// bytes a stage: 256 (e4m3) or 512 (e2m1) values of K.  Against e4m3 rows the
// copy spreads 16 weight codes over 16 bytes, the layout of the mixed kind, so
// HBM and L2 carry 4 bits a weight.  Scales are copied 16 to a row (512 values
// of K, a chunk); four warps move them from shared to tensor memory in the
// MMA's layout (row r in lane r % 32 of every lane quarter, column r / 32),
// several stages ahead.  The row-major scales of a checkpoint can be used as
// they are, and rows of x can start at any row: no 128-row tiling of the
// scales has to fit the segments.
//
// Work: a unit is (expert, 256 weight rows, token tile).  Pairs take whole
// units in turn; what does not fill the last turn is cut along K into equal
// ranges of chunks, one per pair, where that ends sooner (plan()).  The parts of
// a cut unit meet in the workspace: each epilogue warp stores its part of the
// accumulator, and the last of the parts to arrive sums them in K order, so
// the result does not depend on who was last.
//
// Roles per CTA: warp 0 issues the copies, warp 1 of the even CTA the MMAs
// (two to four accumulators), warps 4..7 move scales, warps 8..15 drain the
// accumulators; warp 2 decodes units ahead for all of them and warp 3 copies
// scales.  All waits are bounded.
//
// What bounds it, at the rates of a plain copy (6.54 TB/s) and a bf16 library
// product (1607 TFLOP/s) on the same card.  Times are of 12 calls in a graph;
// behind the slash those of runs of 0.15 s, in which the power cap lowers the
// clock.  Few rows an expert, the weights' bytes and, with e4m3 rows, the issue
// of MMAs (2000 rows over 256 experts of 2048 -> 7168: 353 us, 5.7 TB/s / 407 us,
// 4.9 TB/s; e2m1 rows 297 us, 6.8 TB/s); one token, the latency of a launch's
// ends (14336 -> 4096, 2 experts: 22 us, of which 10 us are the bytes); prefill,
// the operands' way from L2 through shared memory and the power cap (8192 rows,
// 14336 -> 4096: 377 us, 2.6 PFLOP/s / 443 us, 2.2 PFLOP/s; e2m1 rows 198 us,
// 4.9 PFLOP/s; gated 4096 -> 2 x 14336 with e4m3 out: 754 us, 2.6 PFLOP/s /
// 893 us, 2.2 PFLOP/s).
//
// Method: as gemm_pair.cu; the pages' deployment section (jsqmd.com) asks for
// quantised experts.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "gate.cuh"
#include "internal.h"
#include "launch.cuh"
#include "mx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 512;
constexpr int kEpiWarps = 8;
constexpr int kMaxN = 192;               // token rows per tile
constexpr uint32_t kRowBytes = 128;      // of an operand row in shared memory
constexpr uint32_t kATile = 128 * kRowBytes;
constexpr int kChunkK = 512;             // values of K per scale chunk (16 scale bytes)
constexpr uint32_t kScA = 128 * 16;      // bytes of a chunk's weight scales
constexpr int kWorkSlots = 4;            // units announced ahead by the scheduling warp
constexpr int kWorkInts = 16;
constexpr uint32_t kTmemCols = 512;
constexpr int kColChunk = 16;            // accumulator columns per epilogue step
constexpr uint32_t kXchg = 4 * 2 * 2 * 8 * 32 * 4;  // [warp pair][buf][a|b][8][32] fp32
constexpr int kMaxPairs = 80;            // pairs a launch may use (74 on 148 SMs)
constexpr int kParts = 2 * kMaxPairs;    // partial units: two per pair
constexpr size_t kCounters = static_cast<size_t>(kMaxPairs) * 2 * kEpiWarps;

// Layout by the format of x and the largest token tile.  A stage is one step
// of the MMA warp: kAtoms 128-byte columns of both operands, whose MMAs it
// issues in one straight run behind one wait.  (Waits and branches between
// fewer MMAs cost more than the MMAs of a narrow tile: 2000 rows over 256
// experts of 2048 -> 7168, e4m3, 4 MMAs a run 414 us, 8 a run 355 us.)
template <int FMT, int NMAX>
struct Shape {
    static constexpr int kAtoms = 2;
    static constexpr int kAtomK = FMT == kMxE4M3 ? 128 : 256;  // values of K per column
    static constexpr int kStepK = kAtoms * kAtomK;
    static constexpr int kSteps = kChunkK / kStepK;            // per chunk
    static constexpr int kMmas = 4 * kAtoms;                   // per step
    static constexpr int kMmaK = kAtomK / 4;
    static constexpr uint32_t kBTile = NMAX / 2 * kRowBytes;
    static constexpr uint32_t kStage = kAtoms * (kATile + kBTile);
    static constexpr int kStages = (NMAX == 192 ? 6 : 8) / kAtoms;
    static constexpr uint32_t kScSlot = kScA + NMAX * 16;
    static constexpr int kScSlots = 4;  // scale chunks in shared memory
    // Tensor memory: kAccs accumulators of NMAX columns (four where they
    // fit: short units then overlap the latency of several epilogues), then
    // kScBufs buffers of the scales of a step.  128 values of K are one 32-bit
    // word a row: 4 columns of A's scales, then NMAX / 32 of B's.
    static constexpr int kAccs = NMAX == 192 ? 2 : 4;
    static constexpr uint32_t kWord = NMAX == 192 ? 12 : 8;
    static constexpr int kWords = kStepK / 128;
    static constexpr uint32_t kScBuf = kWords * kWord;
    static constexpr uint32_t kScCol = kAccs * NMAX;
    static constexpr int kScBufs = (kTmemCols - kScCol) / kScBuf;
    static_assert(kScBufs >= 2, "tensor memory");
    static constexpr int kBarriers = 2 * kStages + 2 * kScSlots + 2 * kAccs + 2 * kScBufs +
                                     2 * kWorkSlots + 1 + 8;
    static constexpr size_t kBytes = 1024 /* alignment slack */ + kStages * kStage +
                                     kScSlots * kScSlot + kXchg + kBarriers * 8 + 64 +
                                     kWorkSlots * kWorkInts * 4 + 2 * (kMaxE + 1) * sizeof(int32_t);
    static_assert(kBytes <= 227 * 1024, "shared memory");
    static_assert(kBTile % 1024 == 0, "swizzle atom");
    // Rows per copy of x and of its scales: a tile is copied in as many as
    // its columns need.  Few token rows come in small copies, since rows that
    // the MMA does not read take L2 bandwidth from the weights (16 experts of
    // 4096 -> 4096, 8 rows each: 45 us in copies of 48, 40 us in copies of
    // 16) and a copy that reaches beyond the last row of x is slow.
    static constexpr int kXBox = NMAX == 192 ? 96 : 16;
    static constexpr int kXsBox = NMAX == 192 ? 192 : 32;
};

struct GemmParams {
    int S, K, E, N;
    int xbox, xsbox;         // rows per copy of x and its scales
    int rows_blk;            // output columns per unit: 256, or 128 (gated)
    int act, y_type;
    const int32_t *offsets;  // [E+1] or nullptr
    void *y;                 // [S, N] or nullptr
    uint8_t *q, *qs;         // [S, N] e4m3, [S, qpitch]
    int qpitch;
    float *parts;            // [kParts][2 CTAs][part_cols][128 lanes]
    int part_cols;
    uint32_t *ctr;           // kCounters, zero before the launch
    uint32_t *err;
    int own_err;             // the error word is this launch's alone: it resets it
};

// ------------------------------------------------------------------ waiting
// The bounded waits of common.cuh, whose acquire is at CTA scope: what the two
// CTAs hand each other here is shared memory that copies fill and MMAs read,
// and tensor memory, ordered by the tcgen05 fences.
__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity)
{
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (ptx::globaltimer() - t0 > 100000000ull) break;  // 100 ms
    }
}

// --------------------------------------------------------------------- work
__device__ __forceinline__ int ceil16(int v) { return (v + 15) & ~15; }

// A part of a unit: chunks [c0, c1) of K.  When it is not the whole unit, its
// accumulator goes to slot `part` of the workspace and `first` .. `last` are
// the pairs that hold the unit's parts, `cut` the unit's number among those
// that may be cut.
struct Work {
    int e, blk;
    int r0, n;               // the tile's n columns are the rows r0 ..
    int lo, hi;              // of which columns lo .. hi-1 are the unit's
    int c0, c1;
    int part, first, last, cut;
};

// The scheduling warp's announcement of a unit, read by every other role.
__device__ __forceinline__ void put(volatile int32_t *s, const Work &w)
{
    s[0] = w.e;
    s[1] = w.blk;
    s[2] = w.r0;
    s[3] = w.lo;
    s[4] = w.n;
    s[11] = w.hi;
    s[5] = w.c0;
    s[6] = w.c1;
    s[7] = w.part;
    s[8] = w.first;
    s[9] = w.last;
    s[10] = w.cut;
}

__device__ __forceinline__ void get(const int32_t *s, Work &w)
{
    const int v = s[threadIdx.x & 15];
    w.e = __shfl_sync(0xffffffffu, v, 0);
    w.blk = __shfl_sync(0xffffffffu, v, 1);
    w.r0 = __shfl_sync(0xffffffffu, v, 2);
    w.lo = __shfl_sync(0xffffffffu, v, 3);
    w.hi = __shfl_sync(0xffffffffu, v, 11);
    w.n = __shfl_sync(0xffffffffu, v, 4);
    w.c0 = __shfl_sync(0xffffffffu, v, 5);
    w.c1 = __shfl_sync(0xffffffffu, v, 6);
    w.part = __shfl_sync(0xffffffffu, v, 7);
    w.first = __shfl_sync(0xffffffffu, v, 8);
    w.last = __shfl_sync(0xffffffffu, v, 9);
    w.cut = __shfl_sync(0xffffffffu, v, 10);
}

// The sequence of work of one pair; both CTAs walk it alike.
struct Walk {
    int pair, pairs, units, whole, chunks;   // units [whole, units) may be cut
    int cutters;                             // pairs that share those: no range is empty
    int u;                                   // next whole unit
    int it, end, items;                      // chunk items of the cut units (items pairs < 2^20)
    int first_cut;                           // the first cut unit of this pair

    // Units whole, whole + 1, .. hold `items` chunks of K; pair p < cutters
    // has [items p / cutters, items (p + 1) / cutters) of them.
    __device__ __forceinline__ void start(int pair_, int pairs_, int units_, int whole_, int chunks_)
    {
        pair = pair_;
        pairs = pairs_;
        units = units_;
        whole = whole_;
        chunks = chunks_;
        u = pair;
        items = (units - whole) * chunks;
        cutters = items < pairs ? items : pairs;
        it = end = first_cut = 0;
        if (pair < cutters) {
            it = items * pair / cutters;
            end = items * (pair + 1) / cutters;
            first_cut = it / chunks;
        }
    }

    __device__ __forceinline__ int owner(int item) const { return ((item + 1) * cutters - 1) / items; }

    // Next unit and its chunks; false when the pair is done.  Cut units come
    // first, so that whole ones hide the joining of their parts.
    __device__ __forceinline__ bool next(Work &w, int &unit)
    {
        if (it >= end) {
            if (u >= whole) return false;
            unit = u;
            u += pairs;
            w.c0 = 0;
            w.c1 = chunks;
            w.part = -1;
            return true;
        }
        const int c = it / chunks;
        const int base = c * chunks;
        unit = whole + c;
        w.c0 = it - base;
        const int stop = base + chunks < end ? base + chunks : end;
        w.c1 = stop - base;
        it = stop;
        w.part = -1;
        if (w.c0 != 0 || w.c1 != chunks) {
            w.cut = c;
            w.first = owner(base);
            w.last = owner(base + chunks - 1);
            w.part = 2 * pair + (c == first_cut ? 0 : 1);
        }
        return true;
    }

    // The slot in which pair p stores its part of cut unit c.
    __device__ __forceinline__ int part_of(int p, int c) const
    {
        return 2 * p + (items * p / cutters / chunks == c ? 0 : 1);
    }
};

// How many of `units` units of `chunks` chunks are taken whole: all of them,
// or the full turns of the pairs while the rest is cut evenly.  Cutting costs
// storing, waiting for and summing the parts: about 3 us for 16 columns, 10 us
// for 64, 30 us for 176, where a chunk takes about 1 us; it is taken where it
// saves more chunks than that.  Measured: two rows of 14336 -> 4096 (28 chunks
// down to 13) 33.5 us whole, 23.9 us cut; 64 rows of 2048 -> 4096 (4 down to
// 1) 11 us whole, 19 us cut.  The columns charged for are those of the widest
// tile that S rows allow, which the host knows too (it leaves the counters
// uncleared where nothing can be cut), not of the widest that the segments
// have: 64 rows spread one or two to an expert are charged for 64 columns, and
// stay whole up to K = 5632.
__host__ __device__ constexpr int join_chunks(int n) { return 2 + n / 8; }

__device__ __forceinline__ int plan(int units, int pairs, int chunks, int n)
{
    const int full = units / pairs * pairs;
    const int rest = units - full;
    if (rest == 0) return units;
    const int each = (rest * chunks + pairs - 1) / pairs;
    return chunks - each > join_chunks(n) ? full : units;
}

template <int NMAX>
__device__ __forceinline__ int seg_tiles(int cnt) { return (cnt + NMAX - 1) / NMAX; }

// Unit u: expert by the prefix of unit counts, then 256-row block, then tile
// (neighbouring pairs share weights, and the tiles of an expert stay in L2).
template <int NMAX>
__device__ __forceinline__ void place(Work &w, int u, const int32_t *s_off, const int32_t *s_pre,
                                      int E, int S)
{
    int lo = 0, hi = E - 1;
    while (lo < hi) {  // largest e with pre[e] <= u
        const int mid = (lo + hi + 1) >> 1;
        if (s_pre[mid] <= u) lo = mid;
        else hi = mid - 1;
    }
    w.e = lo;
    const int local = u - s_pre[lo];
    const int cnt = s_off[lo + 1] - s_off[lo];
    const int nt = seg_tiles<NMAX>(cnt);
    const int q = ceil16((cnt + nt - 1) / nt);
    w.blk = local / nt;
    const int t = local - w.blk * nt;
    const int first = s_off[lo] + t * q;
    const int rem = cnt - t * q;
    const int valid = rem < 0 ? 0 : rem < q ? rem : q;
    w.n = valid > 0 ? ceil16(valid) : 16;
    // The n columns start earlier where they would reach beyond the last row.
    w.r0 = min(first, max(0, S - w.n));
    w.lo = first - w.r0;
    w.hi = w.lo + valid;
}

__device__ __forceinline__ int warp_scan_incl(int v, int lane)
{
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += n;
    }
    return v;
}

// ----------------------------------------------------------------- epilogue
// NC accumulator columns of 32 lanes to rows t0 .. t0+NC-1 of y in bf16: lane
// pairs swap so that each lane stores two neighbouring output columns.
template <int NC>
__device__ __forceinline__ void store_bf16(const GemmParams &p, const float (&v)[NC], int row,
                                           int t0, int lo, int hi, int o, int lane)
{
    const int odd = lane & 1;
    __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(p.y) + static_cast<size_t>(row + t0) * p.N + (o & ~1);
#pragma unroll
    for (int j = 0; j < NC; j += 2) {
        const float give = odd ? v[j] : v[j + 1];
        const float got = __shfl_xor_sync(0xffffffffu, give, 1);
        const __nv_bfloat162 b = odd ? __floats2bfloat162_rn(got, v[j + 1])
                                     : __floats2bfloat162_rn(v[j], got);
        if (o < p.N && t0 + j + odd >= lo && t0 + j + odd < hi)
            *reinterpret_cast<__nv_bfloat162 *>(y + static_cast<size_t>(j + odd) * p.N) = b;
    }
}

template <int NC>
__device__ __forceinline__ void store_fp32(const GemmParams &p, const float (&v)[NC], int row,
                                           int t0, int lo, int hi, int o)
{
    float *y = static_cast<float *>(p.y) + static_cast<size_t>(row + t0) * p.N + o;
#pragma unroll
    for (int j = 0; j < NC; ++j)
        if (o < p.N && t0 + j >= lo && t0 + j < hi) y[static_cast<size_t>(j) * p.N] = v[j];
}

// Eight tokens of h at 32 columns f (one per lane): bf16, or e4m3 with the
// scale of the 32 lanes.
__device__ __forceinline__ void store_h8(const GemmParams &p, const float (&v)[8], int row, int t0,
                                         int lo, int hi, int f, int lane)
{
    if (p.y != nullptr) {
        const int odd = lane & 1;
        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(p.y) + static_cast<size_t>(row + t0) * p.N + (f & ~1);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float give = odd ? v[j] : v[j + 1];
            const float got = __shfl_xor_sync(0xffffffffu, give, 1);
            const __nv_bfloat162 b = odd ? __floats2bfloat162_rn(got, v[j + 1])
                                         : __floats2bfloat162_rn(v[j], got);
            if (t0 + j + odd >= lo && t0 + j + odd < hi)
                *reinterpret_cast<__nv_bfloat162 *>(y + static_cast<size_t>(j + odd) * p.N) = b;
        }
        return;
    }
    uint32_t amax[8], worst = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        amax[j] = __reduce_max_sync(0xffffffffu, abs_bits(v[j]));
        worst = max(worst, amax[j]);
    }
    uint32_t mine = 0;         // the scale byte of token t0 + lane
    float t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t c = mx_scale_code_finite<kMxE4M3>(amax[j]);
        if (lane == j) mine = c;
        t[j] = v[j] * mx_inv_scale(c);
    }
    uint32_t w[2];             // this lane's codes of tokens 0..3 and 4..7
#pragma unroll
    for (int g = 0; g < 2; ++g)
        w[g] = e4m3x2(t[4 * g], t[4 * g + 1]) | e4m3x2(t[4 * g + 2], t[4 * g + 3]) << 16;
    if (worst >= 0x7f800000u) {  // a token with a NaN or an infinity: codes 0, scale 255
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (amax[j] >= 0x7f800000u) {
                if (lane == j) mine = 255u;
                w[j >> 2] &= ~(0xffu << (8 * (j & 3)));
            }
    }
    if (lane < 8 && t0 + lane >= lo && t0 + lane < hi) {
        uint8_t *s = p.qs + static_cast<size_t>(row + t0 + lane) * p.qpitch;
        s[f >> 5] = static_cast<uint8_t>(mine);
        if ((f >> 5) == (p.N >> 5) - 1)
            for (int b = p.N >> 5; b < p.qpitch; ++b) s[b] = 0;
    }
    // 4 x 4 bytes transposed over groups of four lanes: lane 4i + t gets the
    // codes of columns 4i .. 4i+3 of token t.
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        uint32_t a = w[g];
        uint32_t b = __shfl_xor_sync(0xffffffffu, a, 1);
        a = (lane & 1) ? __byte_perm(a, b, 0x3715) : __byte_perm(a, b, 0x6240);
        b = __shfl_xor_sync(0xffffffffu, a, 2);
        a = (lane & 2) ? __byte_perm(a, b, 0x3276) : __byte_perm(a, b, 0x5410);
        const int tok = t0 + 4 * g + (lane & 3);
        if (tok >= lo && tok < hi)
            *reinterpret_cast<uint32_t *>(p.q + static_cast<size_t>(row + tok) * p.N + (f & ~3)) = a;
    }
}

// ------------------------------------------------------------------- kernel
template <int FMT, bool GATED, int NMAX>
__global__ void __launch_bounds__(kThreads, 1)
    mx_pair_kernel(const __grid_constant__ CUtensorMap tmW1, const __grid_constant__ CUtensorMap tmW3,
                   const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmS1,
                   const __grid_constant__ CUtensorMap tmS3, const __grid_constant__ CUtensorMap tmXs,
                   const GemmParams p)
{
    using SM = Shape<FMT, NMAX>;
    constexpr int kStages = SM::kStages;
    constexpr int kAtoms = SM::kAtoms;
    // e4m3 rows: one copy spreads the weights of a stage's atoms, in groups of
    // 8 rows: [group][atom][8 rows].  e2m1 rows: [atom][rows], a copy each.
    constexpr uint32_t kAGroup = FMT == kMxE4M3 ? kAtoms * 1024 : 1024;
    constexpr uint32_t kAAtom = FMT == kMxE4M3 ? 1024 : kATile;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    // Broadcast, so that the compiler knows them to be the same over a warp:
    // the warps that issue copies and MMAs then keep addresses, descriptors
    // and loop counters in uniform registers, which those instructions read.
    // With one thread's own values every operand was moved over before each
    // MMA: 150 cycles an MMA instead of 97.
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const uint32_t cta = __shfl_sync(0xffffffffu, ptx::cluster_ctarank(), 0);  // 0: issues the MMAs
    const bool leader = (cta == 0);

    uint8_t *scales = smem + kStages * SM::kStage;
    float *xchg = reinterpret_cast<float *>(scales + SM::kScSlots * SM::kScSlot);
    uint64_t *full = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(xchg) + kXchg);
    uint64_t *empty = full + kStages;
    uint64_t *cfull = empty + kStages;      // [kScSlots] scale chunk in shared memory
    uint64_t *cempty = cfull + SM::kScSlots;  // [kScSlots]
    uint64_t *tfull = cempty + SM::kScSlots;  // [kAccs] accumulator
    uint64_t *tempty = tfull + SM::kAccs;   // [kAccs]
    uint64_t *sfull = tempty + SM::kAccs;   // [kScBufs] scales in tensor memory
    uint64_t *sempty = sfull + SM::kScBufs; // [kScBufs]
    uint64_t *wfull = sempty + SM::kScBufs; // [kWorkSlots] unit announced
    uint64_t *wempty = wfull + kWorkSlots;  // [kWorkSlots]
    uint64_t *drain = wempty + kWorkSlots;  // [1]
    uint64_t *xbar = drain + 1;             // [4 warp pairs][2 exchange buffers]
    int32_t *s_work = reinterpret_cast<int32_t *>((reinterpret_cast<uintptr_t>(xbar + 8) + 15) & ~static_cast<uintptr_t>(15));
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(s_work + kWorkSlots * kWorkInts);
    volatile uint32_t *abort_flag = tmem_slot + 1;
    int32_t *s_off = reinterpret_cast<int32_t *>(tmem_slot + 8);
    int32_t *s_pre = s_off + (kMaxE + 1);

    const int E = p.offsets ? p.E : 1;
    const int blocks = (p.N + p.rows_blk - 1) / p.rows_blk;
    const int chunks = (p.K + kChunkK - 1) / kChunkK;
    const int steps = (p.K + SM::kStepK - 1) / SM::kStepK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < SM::kScSlots; ++s) {
            ptx::mbar_init(&cfull[s], 1);
            ptx::mbar_init(&cempty[s], 4);
        }
        for (int b = 0; b < SM::kAccs; ++b) {
            ptx::mbar_init(&tfull[b], 1);
            ptx::mbar_init(&tempty[b], 2 * kEpiWarps);
        }
        for (int b = 0; b < SM::kScBufs; ++b) {
            ptx::mbar_init(&sfull[b], 8);
            ptx::mbar_init(&sempty[b], 1);
        }
        for (int b = 0; b < kWorkSlots; ++b) {
            ptx::mbar_init(&wfull[b], 1);
            // two copying warps, scales, epilogue; the even CTA's MMAs
            ptx::mbar_init(&wempty[b], 2 + 4 + kEpiWarps + (leader ? 1 : 0));
        }
        ptx::mbar_init(drain, 1);
        for (int b = 0; b < 8; ++b) ptx::mbar_init(&xbar[b], 64);
        *abort_flag = 0u;
        ptx::fence_barrier_init();
    }
    if (threadIdx.x == 32) {
        ptx::prefetch_tensormap(&tmW1);
        ptx::prefetch_tensormap(&tmX);
        ptx::prefetch_tensormap(&tmS1);
        ptx::prefetch_tensormap(&tmXs);
        if (GATED) {
            ptx::prefetch_tensormap(&tmW3);
            ptx::prefetch_tensormap(&tmS3);
        }
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(tmem_slot, kTmemCols);
        ptx::tmem_relinquish_pair();
    }
    // Everything above overlaps the previous kernel; from here on its results
    // are read.
    ptx::grid_dep_wait();
    if (warp == 2) {
        // Segment table and the prefix of unit counts per expert.
        const int per = (E + 31) >> 5;
        const int base = lane * per;
        bool bad = false;
        int nu = 0;
        for (int i = 0; i < per; ++i) {
            const int e = base + i;
            if (e < E) {
                const int o0 = p.offsets ? p.offsets[e] : 0;
                const int o1 = p.offsets ? p.offsets[e + 1] : p.S;
                s_off[e] = o0;
                if (e == E - 1) s_off[E] = o1;
                if (o0 < 0 || o1 < o0 || o1 > p.S) bad = true;
                else nu += seg_tiles<NMAX>(o1 - o0) * blocks;
            }
        }
        __syncwarp();
        bad = __any_sync(0xffffffffu, bad);
        if (bad) nu = 0;
        // Every pair sees the same table.  The other bits are set by waits
        // that ran out, seconds after this store.
        if (p.own_err) {
            if (blockIdx.x == 0 && lane == 0) *p.err = bad ? kErrOffsets : 0u;
        } else if (bad && lane == 0 && leader) {
            atomicOr(p.err, kErrOffsets);
        }
        const int incl = warp_scan_incl(nu, lane);
        int run = incl - nu;
        for (int i = 0; i < per; ++i) {
            const int e = base + i;
            if (e < E) {
                s_pre[e] = run;
                if (!bad) run += seg_tiles<NMAX>(s_off[e + 1] - s_off[e]) * blocks;
            }
        }
        if (lane == 31) s_pre[E] = incl;
    }
    // The scheduling warp decodes the pair's first unit before the barrier.
    Work w;
    Walk walk;
    bool more = false;
    const int pairs = static_cast<int>(gridDim.x >> 1);
    if (warp == 2) {
        __syncwarp();
        const int units = s_pre[E];
        walk.start(static_cast<int>(blockIdx.x >> 1), pairs, units, plan(units, pairs, chunks, p.part_cols), chunks);
        if (lane == 0) {
            int unit = 0;
            more = walk.next(w, unit);
            if (more) place<NMAX>(w, unit, s_off, s_pre, E, p.S);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    // Both CTAs' barriers are initialised before either CTA signals the other.
    ptx::cluster_sync();
    ptx::tc_fence_after();
    // Whatever follows may set itself up on SMs that this kernel leaves; it
    // waits for the whole grid before it reads.
    ptx::grid_dep_launch();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    // Shared::cluster addresses of the even CTA's barriers.
    const uint32_t full0 = ptx::mapa_shared(ptx::smem_addr(full), 0);
    const uint32_t tempty0 = ptx::mapa_shared(ptx::smem_addr(tempty), 0);
    const uint32_t sfull0 = ptx::mapa_shared(ptx::smem_addr(sfull), 0);

    // Takes the next announced unit; false at the end (or after a failure).
    uint32_t wslot = 0, wphase = 0;
    auto next_unit = [&]() -> bool {
        if (!bounded_wait_warp(&wfull[wslot], wphase, abort_flag, p.err, kErrTimeoutEpi)) return false;
        get(s_work + wslot * kWorkInts, w);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&wempty[wslot]);
        if (++wslot == kWorkSlots) {
            wslot = 0;
            wphase ^= 1u;
        }
        return w.e >= 0;
    };
    if (warp == 2) {
        // Scheduling: decodes the pair's units ahead of the other roles.
        if (lane == 0) {
            while (true) {
                if (!more) w.e = -1;
                if (!bounded_wait(&wempty[wslot], wphase ^ 1u, abort_flag, p.err, kErrTimeoutEpi)) break;
                put(s_work + wslot * kWorkInts, w);
                ptx::mbar_arrive(&wfull[wslot]);
                if (++wslot == kWorkSlots) {
                    wslot = 0;
                    wphase ^= 1u;
                }
                if (!more) break;
                int unit = 0;
                more = walk.next(w, unit);
                if (more) place<NMAX>(w, unit, s_off, s_pre, E, p.S);
            }
        }
    } else if (warp == 0) {
        const bool one = ptx::elect_one();
        uint32_t stage = 0, phase = 0, issued = 0, last_parity = 0;  // bits by stage
        const uint64_t pol = ptx::policy_evict_normal();
        bool stop = false;
        while (!stop && next_unit()) {
            const int arow = w.e * p.N + w.blk * p.rows_blk + static_cast<int>(cta) * (p.rows_blk / 2);
            const int half = w.n >> 1;
            const int brow = w.r0 + static_cast<int>(cta) * half;
            // Copies of x per atom: in this CTA, and in both.  Fewer than 8
            // rows in all lie in the even CTA's columns.
            const bool few = p.xbox < 8;
            const int nx = few ? 1 - static_cast<int>(cta) : (half + p.xbox - 1) / p.xbox;
            const int nx2 = few ? 1 : 2 * nx;
            const uint32_t tx = kAtoms * (2 * (FMT == kMxE4M3 ? kATile / 2 : kATile) + kRowBytes * p.xbox * nx2);
            const int s1 = min(w.c1 * SM::kSteps, steps);
            for (int st = w.c0 * SM::kSteps; st < s1; ++st) {
                const int a = st * kAtoms;
                if (!bounded_wait_warp(&empty[stage], phase ^ 1u, abort_flag, p.err, kErrTimeoutMma)) {
                    stop = true;
                    break;
                }
                uint8_t *sa = smem + stage * SM::kStage;
                const uint32_t fb = full0 + 8 * stage;
                if (one) {
                    if (leader) ptx::mbar_arrive_expect_tx(&full[stage], tx);
                    // (a spread copy counts the 4-bit codes it moves, not the
                    // shared memory it covers)
                    if constexpr (FMT == kMxE4M3) {
                        ptx::tma_load_4d_pair(sa, &tmW1, fb, 0, 0, a, arow >> 3, pol);
                        if (GATED)
                            ptx::tma_load_4d_pair(sa + kAtoms * kATile / 2, &tmW3, fb, 0, 0, a, arow >> 3, pol);
                    } else {
#pragma unroll
                        for (int t = 0; t < kAtoms; ++t) {
                            uint8_t *at = sa + t * kATile;
                            ptx::tma_load_2d_pair(at, &tmW1, fb, (a + t) * 128, arow, pol);
                            if (GATED) ptx::tma_load_2d_pair(at + kATile / 2, &tmW3, fb, (a + t) * 128, arow, pol);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < kAtoms; ++t)
                        for (int x = 0; x < nx; ++x)
                            ptx::tma_load_2d_pair(sa + kAtoms * kATile + t * SM::kBTile + x * p.xbox * kRowBytes,
                                                  &tmX, fb, (a + t) * 128, brow + x * p.xbox, pol);
                }
                issued |= 1u << stage;
                last_parity = (last_parity & ~(1u << stage)) | phase << stage;
                if (++stage == static_cast<uint32_t>(kStages)) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // No copy may still be landing in shared memory at exit.  The odd
        // CTA's operand copies count on the even CTA's barriers, and the
        // final cluster barrier orders its exit after this.
        if (leader && one)
            for (int s = 0; s < kStages; ++s)
                if (issued & (1u << s)) drain_wait(&full[s], last_parity >> s & 1u);
    } else if (warp == 3) {
        // Copies of scales: few bytes in many short rows, so they take longer
        // than a stage's operands; their own ring runs up to kScSlots chunks
        // ahead.
        const bool one = ptx::elect_one();
        uint32_t slot = 0, cphase = 0, issued = 0, last_parity = 0;
        bool stop = false;
        while (!stop && next_unit()) {
            const int arow = w.e * p.N + w.blk * p.rows_blk + static_cast<int>(cta) * (p.rows_blk / 2);
            const int ns = p.xsbox < SM::kXsBox ? 1 : (w.n + SM::kXsBox - 1) / SM::kXsBox;
            for (int c = w.c0; c < w.c1; ++c) {
                if (!bounded_wait_warp(&cempty[slot], cphase ^ 1u, abort_flag, p.err, kErrTimeoutTma)) {
                    stop = true;
                    break;
                }
                uint8_t *sc = scales + slot * SM::kScSlot;
                if (one) {
                    ptx::mbar_arrive_expect_tx(&cfull[slot], kScA + ns * p.xsbox * 16);
                    ptx::tma_load_2d(sc, &tmS1, &cfull[slot], c * 16, arow);
                    if (GATED) ptx::tma_load_2d(sc + kScA / 2, &tmS3, &cfull[slot], c * 16, arow);
                    for (int x = 0; x < ns; ++x)
                        ptx::tma_load_2d(sc + kScA + x * SM::kXsBox * 16, &tmXs, &cfull[slot], c * 16,
                                         w.r0 + x * SM::kXsBox);
                }
                issued |= 1u << slot;
                last_parity = (last_parity & ~(1u << slot)) | cphase << slot;
                if (++slot == SM::kScSlots) {
                    slot = 0;
                    cphase ^= 1u;
                }
            }
        }
        if (one)
            for (int s = 0; s < SM::kScSlots; ++s)
                if (issued & (1u << s)) drain_wait(&cfull[s], last_parity >> s & 1u);
    } else if (warp == 1) {
        if (leader) {
            const bool one = ptx::elect_one();
            uint32_t stage = 0, phase = 0, sb = 0, sphase = 0;
            // Descriptors differ in their start address (16-byte units) only.
            const uint64_t desc_a = ptx::sw128_kmajor_desc(0, kAGroup);
            const uint64_t desc_b = ptx::sw128_kmajor_desc(0);
            const uint32_t smem16 = ptx::smem_addr(smem) >> 4;
            const uint32_t fmt_a = FMT == kMxE4M3 ? ptx::kMxf8f6f4E2M1 : ptx::kMxf4E2M1;
            const uint32_t fmt_b = FMT == kMxE4M3 ? ptx::kMxf8f6f4E4M3 : ptx::kMxf4E2M1;
            bool stop = false;
            for (uint32_t i = 0; !stop && next_unit(); ++i) {
                const uint32_t buf = i % SM::kAccs;
                const uint32_t idesc = ptx::idesc_mx(256, w.n, fmt_a, fmt_b, 0);
                if (!bounded_wait_warp(&tempty[buf], ((i / SM::kAccs) & 1u) ^ 1u, abort_flag, p.err, kErrTimeoutEpi))
                    break;
                ptx::tc_fence_after();
                const uint32_t dacc = tmem + buf * NMAX;
                uint32_t acc = 0;
                // One MMA of a step: column t = m / 4 of the operands, 32 bytes
                // of its rows.  e4m3 rows: 32 values, byte kk of the column's
                // word of scales.  e2m1 rows: 64 values, two bytes of the
                // first or second of the column's two words.
                auto mma = [&](int m, uint32_t a16, uint32_t word0, uint32_t accumulate) {
                    const int t = m >> 2, kk = m & 3;
                    const uint64_t da = desc_a | (a16 + t * (kAAtom >> 4));
                    const uint64_t db = desc_b | (a16 + ((kAtoms * kATile + t * SM::kBTile) >> 4));
                    if constexpr (FMT == kMxE4M3) {
                        const uint32_t word = word0 + SM::kWord * t;
                        ptx::tc_mma_mxf8f6f4_pair(dacc, da + 2 * kk, db + 2 * kk, idesc + ptx::idesc_mx_sf(kk),
                                                  word, word + 4, accumulate);
                    } else {
                        const uint32_t word = word0 + SM::kWord * (2 * t + (kk >> 1));
                        ptx::tc_mma_mxf4_pair(dacc, da + 2 * kk, db + 2 * kk,
                                              idesc + ptx::idesc_mx_sf(2 * (kk & 1)), word, word + 4, accumulate);
                    }
                };
                const int s1 = min(w.c1 * SM::kSteps, steps);
                for (int st = w.c0 * SM::kSteps; st < s1; ++st) {
                    if (!bounded_wait_warp(&sfull[sb], sphase, abort_flag, p.err, kErrTimeoutTma) ||
                        !bounded_wait_warp(&full[stage], phase, abort_flag, p.err, kErrTimeoutTma)) {
                        stop = true;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t a16 = smem16 + stage * (SM::kStage >> 4);
                    const uint32_t word0 = tmem + SM::kScCol + sb * SM::kScBuf;
                    const int left = (p.K - st * SM::kStepK) / SM::kMmaK;  // MMAs up to the end of K
                    if (one) {
                        if (left >= SM::kMmas) {
#pragma unroll
                            for (int m = 0; m < SM::kMmas; ++m) mma(m, a16, word0, m ? 1u : acc);
                        } else {
#pragma unroll
                            for (int m = 0; m < SM::kMmas; ++m)
                                if (m < left) mma(m, a16, word0, m ? 1u : acc);
                        }
                        ptx::tc_commit_pair(&empty[stage], 0x3);
                        ptx::tc_commit_pair(&sempty[sb], 0x3);
                    }
                    acc = 1;
                    if (++stage == static_cast<uint32_t>(kStages)) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++sb == static_cast<uint32_t>(SM::kScBufs)) {
                        sb = 0;
                        sphase ^= 1u;
                    }
                }
                if (!stop && one) ptx::tc_commit_pair(&tfull[buf], 0x3);
            }
            // Every MMA issued above has finished once this arrives.
            if (one) {
                ptx::tc_commit_pair(drain, 0x1);
                drain_wait(drain, 0u);
            }
        }
    } else if (warp >= 4 && warp < 8) {
        // Scales: shared memory (row-major, 16 bytes a row) to this warp's
        // lane quarter of tensor memory.
        const uint32_t tq = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + SM::kScCol;
        constexpr int kB = NMAX / 32;
        uint32_t slot = 0, cphase = 0, sb = 0, sphase = 0;
        bool stop = false;
        while (!stop && next_unit()) {
            for (int c = w.c0; c < w.c1 && !stop; ++c) {
                if (!bounded_wait_warp(&cfull[slot], cphase, abort_flag, p.err, kErrTimeoutTma)) {
                    stop = true;
                    break;
                }
                const uint4 *src = reinterpret_cast<const uint4 *>(scales + slot * SM::kScSlot);
                uint4 a[4], b[kB];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = src[32 * i + lane];
#pragma unroll
                for (int i = 0; i < kB; ++i) b[i] = src[128 + 32 * i + lane];
                const uint32_t used = slot;
                if (++slot == SM::kScSlots) {
                    slot = 0;
                    cphase ^= 1u;
                }
#pragma unroll
                for (int h = 0; h < SM::kSteps; ++h) {
                    if (SM::kSteps * c + h >= steps) break;
                    if (!bounded_wait_warp(&sempty[sb], sphase ^ 1u, abort_flag, p.err, kErrTimeoutMma)) {
                        stop = true;
                        break;
                    }
                    ptx::tc_fence_after();
                    uint32_t r[SM::kScBuf];
#pragma unroll
                    for (int j = 0; j < SM::kWords; ++j)
#pragma unroll
                        for (int i = 0; i < static_cast<int>(SM::kWord); ++i) {
                            uint32_t v = 0u;
                            if (i < 4) v = reinterpret_cast<const uint32_t *>(&a[i])[SM::kWords * h + j];
                            else if (i - 4 < kB) v = reinterpret_cast<const uint32_t *>(&b[i - 4])[SM::kWords * h + j];
                            r[SM::kWord * j + i] = v;
                        }
                    const uint32_t dst = tq + sb * SM::kScBuf;
#pragma unroll
                    for (int z = 0; z + 16 <= static_cast<int>(SM::kScBuf); z += 16)
                        ptx::tmem_st16(dst + z, *reinterpret_cast<const uint32_t(*)[16]>(&r[z]));
                    if constexpr (SM::kScBuf % 16 != 0)
                        ptx::tmem_st8(dst + SM::kScBuf - 8, *reinterpret_cast<const uint32_t(*)[8]>(&r[SM::kScBuf - 8]));
                    ptx::tc_wait_st();
                    ptx::tc_fence_before();
                    __syncwarp();
                    // The slot is free only now that the loads' results have
                    // been used: an arrival does not wait for the loads before
                    // it, and the next copy then overtook them (seen as rare
                    // wrong scales in one lane quarter).
                    if (h == 0 && lane == 0) ptx::mbar_arrive(&cempty[used]);
                    if (lane == 0) ptx::mbar_arrive_pair(sfull0 + 8 * sb);
                    if (++sb == static_cast<uint32_t>(SM::kScBufs)) {
                        sb = 0;
                        sphase ^= 1u;
                    }
                }
            }
        }
    } else if (warp >= 8) {
        // Epilogue: warp w reads tensor-memory lanes 32*(w%4)..+31; the two
        // warps of a lane quarter take alternate chunks of 16 columns.
        const int q = warp & 3;
        const int half = (warp - 8) >> 2;
        const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
        const int wpair = (q & 1) + 2 * half;  // (a, b) warp pairs: quarters (0,2) and (1,3)
        const bool is_a = q < 2;               // lanes 0..63: W1 products (gated)
        // for the slots of other pairs' parts
        walk.start(static_cast<int>(blockIdx.x >> 1), pairs, s_pre[E], plan(s_pre[E], pairs, chunks, p.part_cols), chunks);
        float *xa = xchg + wpair * (2 * 2 * 8 * 32);
        uint32_t xuse[2] = {0u, 0u};
        int xb = 0;
        bool stop = false;
        for (uint32_t i = 0; !stop && next_unit(); ++i) {
            const uint32_t buf = i % SM::kAccs;
            if (!bounded_wait_warp(&tfull[buf], (i / SM::kAccs) & 1u, abort_flag, p.err, kErrTimeoutMma)) break;
            ptx::tc_fence_after();
            // The two warps of a quarter swap roles from unit to unit, so that
            // units of one chunk keep both busy.
            const int turn = half ^ static_cast<int>(i & 1u);
            const uint32_t tb = tmem + lane_base + buf * NMAX;
            const int nch = w.n / kColChunk;
            // output column of this lane: product, or h of the lane's quarter
            const int o = GATED ? w.blk * 128 + static_cast<int>(cta) * 64 + (q & 1) * 32 + lane
                                : w.blk * 256 + static_cast<int>(cta) * 128 + 32 * q + lane;
            const size_t pstep = static_cast<size_t>(p.part_cols) * 128;  // one CTA's part
            if (w.part >= 0) {
                float *dst = p.parts + (static_cast<size_t>(w.part) * 2 + cta) * pstep + 32 * q + lane;
                for (int c = turn; c < nch; c += 2) {
                    uint32_t r[16];
                    ptx::tmem_ld16(tb + static_cast<uint32_t>(c * kColChunk), r);
                    ptx::tc_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        __stcg(dst + static_cast<size_t>(c * kColChunk + j) * 128, __uint_as_float(r[j]));
                }
            } else {
                for (int c = turn; c < nch; c += 2) {
                    uint32_t r[16];
                    ptx::tmem_ld16(tb + static_cast<uint32_t>(c * kColChunk), r);
                    ptx::tc_wait_ld();
                    if constexpr (GATED) {
                        // a warps keep tokens 0..7 of the chunk and hand 8..15
                        // to their b partner; b warps the other way round.
                        float *mine = xa + xb * (2 * 8 * 32) + (is_a ? 0 : 8 * 32) + lane;
                        float *theirs = xa + xb * (2 * 8 * 32) + (is_a ? 8 * 32 : 0) + lane;
                        if (is_a) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) mine[j * 32] = __uint_as_float(r[8 + j]);
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j) mine[j * 32] = __uint_as_float(r[j]);
                        }
                        ptx::mbar_arrive(&xbar[wpair * 2 + xb]);
                        const bool okx = bounded_wait(&xbar[wpair * 2 + xb], xuse[xb] & 1u, abort_flag,
                                                      p.err, kErrTimeoutEpi);
                        ++xuse[xb];
                        if (!__all_sync(0xffffffffu, okx)) {
                            stop = true;
                            break;
                        }
                        const int t0 = c * kColChunk + (is_a ? 0 : 8);
                        float v[8], most = 0.0f;
                        if (is_a) {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                v[j] = gate_mul(__uint_as_float(r[j]), theirs[j * 32], p.act, most);
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                v[j] = gate_mul(theirs[j * 32], __uint_as_float(r[8 + j]), p.act, most);
                        }
                        if (__any_sync(0xffffffffu, most >= kGateRange)) {
                            // results take the place of the partner's values,
                            // which only this lane reads
#pragma unroll 1
                            for (int j = 0; j < 8; ++j) {
                                const float own = __uint_as_float(ptx::tmem_ld1(tb + static_cast<uint32_t>(t0 + j)));
                                ptx::tc_wait_ld();
                                const float got = theirs[j * 32];
                                theirs[j * 32] = gate_redo(is_a ? own : got, is_a ? got : own, p.act);
                            }
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[j] = theirs[j * 32];
                        }
                        store_h8(p, v, w.r0, t0, w.lo, w.hi, o, lane);
                        xb ^= 1;
                    } else {
                        float v[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
                        if (p.y_type == kTypeBf16) store_bf16<16>(p, v, w.r0, c * kColChunk, w.lo, w.hi, o, lane);
                        else store_fp32<16>(p, v, w.r0, c * kColChunk, w.lo, w.hi, o);
                    }
                }
                if (stop) break;
            }
            // The accumulator may be reused once every epilogue warp of both
            // CTAs has read it.
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader) ptx::mbar_arrive(&tempty[buf]);
                else ptx::mbar_arrive_pair(tempty0 + 8 * buf);
            }
            if (w.part >= 0) {
                // The last warp to arrive (of the warp's own columns and
                // lanes; gated: of the pair of warps with both sums) adds the
                // parts in K order.
                __threadfence();
                __syncwarp();
                uint32_t seen = 0;
                uint32_t *ctr = p.ctr + (static_cast<size_t>(w.cut) * 2 + cta) * kEpiWarps +
                                (GATED ? (q & 1) + 2 * turn : q + 4 * turn);
                if (lane == 0) seen = atomicAdd(ctr, 1u);
                seen = __shfl_sync(0xffffffffu, seen, 0);
                const uint32_t all = static_cast<uint32_t>(w.last - w.first + 1) * (GATED ? 2u : 1u);
                if (seen + 1 == all) {
                    __threadfence();
                    const float *base = p.parts + cta * pstep + lane + 32 * (GATED ? (q & 1) : q);
                    for (int c = turn; c < nch; c += 2) {
                        for (int h8 = 0; h8 < 16 && c * kColChunk + h8 < w.hi; h8 += 8) {
                            float v[8], u[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[j] = u[j] = 0.0f;
                            // four parts' loads in flight together
                            for (int pr = w.first; pr <= w.last; pr += 4) {
                                float a[4][8], b[4][8];
#pragma unroll
                                for (int g = 0; g < 4; ++g) {
                                    const bool has = pr + g <= w.last;
                                    const float *src =
                                        base + static_cast<size_t>(has ? walk.part_of(pr + g, w.cut) : 0) * 2 * pstep +
                                        static_cast<size_t>(c * kColChunk + h8) * 128;
#pragma unroll
                                    for (int j = 0; j < 8; ++j) {
                                        a[g][j] = has ? __ldcg(src + j * 128) : 0.0f;
                                        if (GATED) b[g][j] = has ? __ldcg(src + j * 128 + 64) : 0.0f;
                                    }
                                }
#pragma unroll
                                for (int g = 0; g < 4; ++g)
#pragma unroll
                                    for (int j = 0; j < 8; ++j) {
                                        v[j] += a[g][j];
                                        if (GATED) u[j] += b[g][j];
                                    }
                            }
                            if constexpr (GATED) {
#pragma unroll
                                for (int j = 0; j < 8; ++j) v[j] = gate_redo(v[j], u[j], p.act);
                                store_h8(p, v, w.r0, c * kColChunk + h8, w.lo, w.hi, o, lane);
                            } else if (p.y_type == kTypeBf16) {
                                store_bf16<8>(p, v, w.r0, c * kColChunk + h8, w.lo, w.hi, o, lane);
                            } else {
                                store_fp32<8>(p, v, w.r0, c * kColChunk + h8, w.lo, w.hi, o);
                            }
                        }
                    }
                }
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    // Neither CTA may free tensor memory or exit while the other still
    // signals its barriers or reads the accumulators.
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, kTmemCols);
    }
    ptx::cluster_sync();
}

// Clusters of two that fit the device at a time, per kernel (0: the kernel
// cannot run here); the first call on a device also sets the kernel up.
template <int FMT, bool GATED, int NMAX>
int pair_count(cudaLaunchConfig_t &cfg)
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    const cudaError_t e = cudaFuncSetAttribute(mx_pair_kernel<FMT, GATED, NMAX>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(cfg.dynamicSmemBytes));
    if (e != cudaSuccess) return 0;
    if (cudaOccupancyMaxActiveClusters(&n, mx_pair_kernel<FMT, GATED, NMAX>, &cfg) != cudaSuccess || n < 1)
        n = device_sm_count() / 2;
    n = std::max(1, std::min(n, kMaxPairs));
    known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Columns of the widest tile.
int part_cols(int S, int nmax) { return std::min(nmax, (S + 15) / 16 * 16); }

template <int FMT, bool GATED, int NMAX>
cudaError_t launch_t(const MxGemmLaunch &a, cudaStream_t s)
{
    using SM = Shape<FMT, NMAX>;
    const uint64_t wrows = static_cast<uint64_t>(a.E) * a.N;
    const uint32_t abox = GATED ? 64 : 128;
    const int xbox = a.S < 8 ? a.S : a.S < SM::kXBox ? 8 : SM::kXBox;
    const int xsbox = std::min(SM::kXsBox, a.S);
    const int nsc = a.K / kMxBlock, wsc = mx_scale_pitch(a.K);
    CUtensorMap tW1, tW3, tX, tS1, tS3, tXs;
    auto weights = [&](CUtensorMap *m, const uint8_t *w) {
        return FMT == kMxE4M3 ? make_tmap_e2m1_wide(m, w, wrows, a.K, abox, SM::kAtoms)
                              : make_tmap_rows(m, w, wrows, a.K / 2, a.K / 2, 128, abox);
    };
    cudaError_t e = weights(&tW1, a.W1);
    if (e == cudaSuccess) e = make_tmap_rows(&tS1, a.s1, wrows, nsc, wsc, 16, abox);
    if (GATED) {
        if (e == cudaSuccess) e = weights(&tW3, a.W3);
        if (e == cudaSuccess) e = make_tmap_rows(&tS3, a.s3, wrows, nsc, wsc, 16, abox);
    } else {
        tW3 = tW1;
        tS3 = tS1;
    }
    if (e == cudaSuccess)
        e = make_tmap_rows(&tX, a.x, a.S, FMT == kMxE4M3 ? a.K : a.K / 2, a.x_stride, 128, xbox);
    if (e == cudaSuccess) e = make_tmap_rows(&tXs, a.xs, a.S, nsc, a.xs_stride, 16, xsbox);
    if (e != cudaSuccess) return e;
    auto *kernel = mx_pair_kernel<FMT, GATED, NMAX>;
    GemmParams p{};
    p.S = a.S;
    p.K = a.K;
    p.E = a.E;
    p.N = a.N;
    p.xbox = xbox;
    p.xsbox = xsbox;
    p.rows_blk = GATED ? 128 : 256;
    p.act = a.act;
    p.y_type = a.y_type;
    p.offsets = a.offsets;
    p.y = a.y;
    p.q = a.q;
    p.qs = a.qs;
    p.qpitch = mx_scale_pitch(a.N);
    p.ctr = reinterpret_cast<uint32_t *>(a.counters);
    p.parts = reinterpret_cast<float *>(a.scratch);
    p.part_cols = part_cols(a.S, NMAX);
    p.err = a.err;
    p.own_err = a.own_err ? 1 : 0;

    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = SM::kBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(2);
    const int pairs = pair_count<FMT, GATED, NMAX>(cfg);
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.numAttrs = a.pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, tW1, tW3, tX, tS1, tS3, tXs, p);
}

// Largest token tile of a launch.
int tile_rows(const MxGemmLaunch &a)
{
    // Rows per expert if they were even.  16 experts of 4096 -> 4096 with
    // uneven segments, e4m3 rows, tiles of at most 96 / 192 rows: 8 rows an
    // expert 40 / 47 us, 32: 41 / 45, 64: 42 / 44, 80: 50 / 45, 96: 55 / 45.
    // The number of units does not enter: a few wide segments of narrow
    // weights (777 rows over 4 experts of 1408 -> 1000: 24 units) leave pairs
    // idle.
    const int rows = (a.S + a.E - 1) / a.E;
    return rows <= 64 ? 96 : kMaxN;
}

template <int FMT, bool GATED>
cudaError_t launch_n(const MxGemmLaunch &a, cudaStream_t s)
{
    if (tile_rows(a) == 96) return launch_t<FMT, GATED, 96>(a, s);
    return launch_t<FMT, GATED, kMaxN>(a, s);
}

}  // namespace

// Zeroes the header and counters of a workspace ahead of a product.  A kernel
// and not a memset, so that the product's set-up overlaps it.
__global__ void __launch_bounds__(512) clear_kernel(uint4 *p, int n)
{
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    for (int i = threadIdx.x; i < n; i += 512) p[i] = make_uint4(0u, 0u, 0u, 0u);
}

cudaError_t launch_clear(void *p, size_t bytes, cudaStream_t s)
{
    return launch_pdl(clear_kernel, dim3(1), dim3(512), 0, s, true, static_cast<uint4 *>(p),
                      static_cast<int>(bytes / 16));
}

size_t mx_gemm_zero_bytes() { return kCounters * sizeof(uint32_t); }

size_t mx_gemm_scratch_bytes(int S)
{
    return static_cast<size_t>(kParts) * 2 * 128 * part_cols(S, kMaxN) * sizeof(float);
}

bool mx_gemm_needs_counters(const MxGemmLaunch &a)
{
    // plan() leaves every unit whole when even one chunk a pair saves too little
    const int chunks = (a.K + kChunkK - 1) / kChunkK;
    return chunks - 1 > join_chunks(part_cols(a.S, tile_rows(a)));
}

cudaError_t launch_mx_gemm(const MxGemmLaunch &a, cudaStream_t s)
{
    if (a.fmt == kMxE4M3) return a.W3 ? launch_n<kMxE4M3, true>(a, s) : launch_n<kMxE4M3, false>(a, s);
    return a.W3 ? launch_n<kMxE2M1, true>(a, s) : launch_n<kMxE2M1, false>(a, s);
}

}  // namespace moe
