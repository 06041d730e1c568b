// attention_prefill.cu -- causal attention of packed sequences with grouped
// heads on the sm_100a tensor cores: whole prompts, pieces of prompts behind a
// cached past, single tokens of many requests.
//
// "How to Run BitNet Inference on GPU Using CUDA Kernels: A Complete Guide",
// section "Understanding the Two-Phase Architecture" (the prefill phase runs
// Attention over the whole prompt).
//
// Mathematics.  For a block of keys with scores S = q K^T (fp32), a reference
// maximum m and c = scale * log2(e):
//   P = 2^(c S - c m),  l <- l + sum P,  O <- O + P V
// m starts as the first block's maximum and moves only when a later block's
// exceeds it by more than 8 / c: then O and l are multiplied by 2^(c (m - m')).
// Until then P stays below 2^8, which fp32 sums and bf16 weights hold as well
// as values below 1, and the pass over O is saved.  out = O / l.
//
// Rows.  The query heads of a kv head share its keys, so a tile's 128 rows are
// (token, head of the group): TM = 128 / G tokens of G heads.  A tile of one
// token and a long cache is then G rows against one pass over the keys, and a
// prompt's tile spans few tokens, so little of its last key blocks is masked.
//
// Two streams.  A CTA keeps two rows of products going, each with its own S
// and O in tensor memory (4 x 128 columns), its own four softmax warps (a
// thread per row), and P written over S as the next product's operand:
//   pair  two tiles of rows share every key block (prompts: each block of K
//         and V is read once for 256 rows);
//   alt   one tile, key blocks alternate between the streams, whose results
//         are merged at the end (few rows: two blocks are in flight).
// While one stream's warps compute exponentials, the tensor cores run the
// other's products.
//
// Work.  The key blocks of all tiles form one line; CTA c takes the c-th of
// equal parts of it, whatever the sequences' lengths.  A tile that is cut has
// its parts' O, m and l (fp32) in the workspace, and a second kernel joins
// them in order.  Each CTA cuts at most two tiles, one at either end.
//
// Warp roles (384 threads; warp 11 idles):
//   warps 0-3, 4-7  softmax of streams 0 and 1, a row per thread; epilogue
//   warp 8          work list and TMA loads (Q, then K and V blocks in a ring)
//   warp 9          MMA issue (lane 0, the whole warp in uniform control flow),
//                   the streams in turn
//   warp 10         values behind a mask: in blocks where some row's keys are
//                   masked, non-finite values of V are zeroed before the
//                   product (a zero weight times a NaN would reach rows that
//                   do not see it) and rows that do see them get NaN.
//
// Measured (20 + 5 heads, with the join; a graph of nine calls): a prompt of 8192
// 296 to 303 us, 1.13 to 1.16 PFLOP/s (tensor pipe 54% active, exponentials 57%: the
// hand-off from products to exponentials and back bounds it, each stream filling
// the other's gaps); 12 packed prompts of up to 1301 93 us; 509 tokens behind 3500
// 35 us; a token each of 64 requests with up to 4096 keys 71 us, 5.1 TB/s; 16 + 2
// heads, a token after 30000 18 us; a prompt of 37 8.7 us.  Repeated for seconds, at
// the clocks that the power limit leaves: 347 us, 0.99 PFLOP/s, for the prompt of
// 8192 and 77 to 81 us, 4.5 to 4.7 TB/s, for the 64 requests.
//
// Every mbarrier wait is bounded (2 s); on expiry BL_ERR_TIMEOUT is recorded,
// every role leaves its loop, copies and MMAs in flight drain, tensor memory
// is freed and the CTA returns.
#include <algorithm>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "tcgen05_common.cuh"

namespace bl {
namespace {

constexpr int kHD = 128;                  // head dimension
constexpr int kRows = 128;                // rows per tile (MMA M)
constexpr int kKeys = 128;                // keys per block (MMA N of the scores)
constexpr int kThreads = 384;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kFixWarp = 10;
constexpr uint32_t kBox = 128 * 128;      // 64 columns x 128 rows of bf16, one swizzle span wide
constexpr uint32_t kTile = 2 * kBox;      // 128 x 128 bf16
constexpr int kItems = 4;                 // work list ring
constexpr int kTileExtra = 2;             // what a tile costs besides its key blocks, in key blocks
constexpr float kRescale = 8.0f;          // log2 of the growth of a row's weights before O is rescaled
// Registers: 168 a thread at launch; a softmax thread holds its row of S.  They
// leave no room on an SM for a CTA of the kernel before this one, so a kernel that
// lets its dependents start before it allocates tensor memory (gemv_tc.cu) never
// finds all of it taken here by a CTA that waits for that kernel's end.
constexpr int kSoftmaxRegs = 200, kOtherRegs = 104;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "register split");

// Instruction descriptors: D fp32, A and B bf16, M = N = 128; B is K-major for
// the scores (keys x dimensions) and MN-major for the values (the same tile,
// dimensions as N).
constexpr uint32_t kIdescQK = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(kKeys >> 3) << 17) |
                              (uint32_t(kRows >> 4) << 24);
constexpr uint32_t kIdescPV = kIdescQK | (1u << 16);

template <bool PAIR>
constexpr int kv_stages() { return PAIR ? 5 : 6; }

// One piece of work: key blocks [j0, j1) of a tile of rows.
struct Item {
    int valid;
    int kvh;                // kv head
    int q_row, toks;        // first row of q and tokens of the tile
    int lim0, nk;           // token i of the tile sees the keys below min(nk, lim0 + i)
    int k_row;              // first key row of the sequence
    int j0, n;              // first key block, number of blocks (0: no row sees a key)
    int nb[2];              // blocks of each stream
    int slot;               // workspace slot, -1: the tile is whole
};

// What the joining kernel needs about the tile whose first part a CTA holds.
struct alignas(16) JoinHeader {
    int valid;
    int kvh, q_row, toks;
    int last;               // CTA of the last part
    int pad[3];
};

struct PrefillParams {
    __nv_bfloat16 *out;
    int64_t o_row, o_head;
    const int32_t *cu_q, *cu_k;
    int batch, Hkv, G, TM;
    int64_t Tq, Tk;
    float c;                // scale * log2(e)
    JoinHeader *hdr;        // [grid]
    float *part_o;          // [2 * grid][rows][128]
    float2 *part_ml;        // [2 * grid][rows]
    int *status;
};

template <bool PAIR>
struct Smem {
    static constexpr int kStages = kv_stages<PAIR>();
    static constexpr int kQTiles = PAIR ? 2 : 1;
    unsigned char q[kQTiles][kTile];
    unsigned char kv[kStages][kTile];
    uint64_t kv_full[kStages], kv_empty[kStages];
    uint64_t v_posted[kStages];      // a block that needs fixing has been asked for in this stage
    uint64_t v_fixed[kStages];
    uint64_t q_full, q_empty;
    uint64_t s_full[2];      // scores complete (and every earlier product)
    uint64_t p_full[2];      // weights written over the scores
    uint64_t o_full[2];      // last product of the piece complete
    uint64_t ml_full;        // alt: stream 1's m and l are in ml
    uint64_t o1_read;        // alt: stream 1's O has been read
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t drain;
    Item item[kItems];
    float2 ml[PAIR ? 1 : kRows];
    int poison_piece;        // piece that poison is about
    int poison[kHD];         // first key with a non-finite value in this dimension
    uint32_t tmem_base;
    int abort_flag;
};

template <bool PAIR>
constexpr uint32_t smem_bytes() { return uint32_t(sizeof(Smem<PAIR>)); }
static_assert(smem_bytes<true>() <= 227 * 1024 && smem_bytes<false>() <= 227 * 1024, "shared memory per CTA");
static_assert(smem_bytes<true>() > 114 * 1024 && smem_bytes<false>() > 114 * 1024,
              "one CTA per SM: it owns all of the tensor memory");

// ---------------------------------------------------------------- PTX wrappers

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2,
                                            int c3)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// K-major and MN-major operands share the stride between 8-row groups; the
// latter also has a stride between its 64-column boxes.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t addr)
{
    return (smem_desc_sw128(addr) & ~(uint64_t(0x3fff) << 16)) | (uint64_t(kBox >> 4) << 16);
}

// Scores of one key block: eight MMAs over the 128 dimensions, operands in
// shared memory, four in each 64-column box.
__device__ __forceinline__ void mma_scores(uint32_t d, uint64_t a, uint64_t b)
{
    constexpr uint32_t box = kBox >> 4;
    asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b32 r;\n\t"
        "mov.u32 r, %%laneid;\n\t"
        "setp.eq.u32 e, r, 0;\n\t"
        "setp.ne.b32 p, %18, %18;\n\t"
        "setp.eq.b32 t, %18, %18;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %9, %17, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %2, %10, %17, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %3, %11, %17, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %4, %12, %17, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %5, %13, %17, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %6, %14, %17, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %7, %15, %17, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %8, %16, %17, t;\n\t}" ::"r"(d),
        "l"(a), "l"(a + 2), "l"(a + 4), "l"(a + 6), "l"(a + box), "l"(a + box + 2), "l"(a + box + 4),
        "l"(a + box + 6), "l"(b), "l"(b + 2), "l"(b + 4), "l"(b + 6), "l"(b + box), "l"(b + box + 2),
        "l"(b + box + 4), "l"(b + box + 6), "r"(kIdescQK), "r"(0u)
        : "memory");
}

// Weights (tensor memory) times values: eight MMAs over the 128 keys, 16 keys
// (two 8-row groups, 2048 bytes) each.
__device__ __forceinline__ void mma_values(uint32_t d, uint32_t a, uint64_t b, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b32 r;\n\t"
        "mov.u32 r, %%laneid;\n\t"
        "setp.eq.u32 e, r, 0;\n\t"
        "setp.ne.b32 p, %18, 0;\n\t"
        "setp.eq.b32 t, %18, %18;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %9, %17, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], %10, %17, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], %11, %17, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%4], %12, %17, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%5], %13, %17, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%6], %14, %17, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%7], %15, %17, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%8], %16, %17, t;\n\t}" ::"r"(d),
        "r"(a), "r"(a + 8), "r"(a + 16), "r"(a + 24), "r"(a + 32), "r"(a + 40), "r"(a + 48), "r"(a + 56), "l"(b),
        "l"(b + 128), "l"(b + 256), "l"(b + 384), "l"(b + 512), "l"(b + 640), "l"(b + 768), "l"(b + 896),
        "r"(kIdescPV), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Pairs of fp32 values in one register pair.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// The weights of one row's scores, written over them as bf16; returns their
// sum.  Two exponentials, one packed multiply-add, one packed sum and one
// conversion a pair: 128 exponentials take 1024 cycles of a quarter SM's unit
// (4 a clock), about what the tensor cores need for the other stream.  A
// cubic on the FMA pipe for every 4th pair took that unit's load down and the
// 8192-token prompt from 343 to 363 us up: the issue slots are the scarcer.
__device__ __forceinline__ float row_weights(const uint32_t (&v)[128], float c, float mc, uint32_t s_tmem)
{
    const uint64_t c2 = pack_f32x2(c, c), m2 = pack_f32x2(-mc, -mc);
    uint64_t sum[2] = {0, 0};       // two pairs of zeros
    uint32_t w[2][32];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int x = 0; x < 32; ++x) {
            const int e = 64 * h + 2 * x;
            float a, b;
            unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), c2, m2), a, b);
            a = exp2_approx(a);
            b = exp2_approx(b);
            sum[x & 1] = add_f32x2(sum[x & 1], pack_f32x2(a, b));
            w[h][x] = bf16x2(a, b);
        }
        tmem_st32(s_tmem + uint32_t(32 * h), w[h]);
    }
    tmem_wait_st();
    tmem_keep32(w[0]);
    tmem_keep32(w[1]);
    float s0, s1;
    unpack_f32x2(add_f32x2(sum[0], sum[1]), s0, s1);
    return s0 + s1;
}

// Thirty-two bytes in one store where the address allows it: a row's stores
// lie 32 lanes apart, and each costs a cache line per lane.
__device__ __forceinline__ void store32(void *dst, const uint32_t (&w)[8], bool aligned)
{
    if (aligned)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    else {
        static_cast<uint4 *>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// ---------------------------------------------------------------- the work line

// Bounds of sequence b; false if they are not ascending and within the rows.
__device__ __forceinline__ bool sequence(const PrefillParams &p, int b, int &q0, int &nq, int &k0, int &nk)
{
    q0 = int(ld_dep_u32(p.cu_q + b));
    const int q1 = int(ld_dep_u32(p.cu_q + b + 1));
    k0 = int(ld_dep_u32(p.cu_k + b));
    const int k1 = int(ld_dep_u32(p.cu_k + b + 1));
    const bool ok = q0 >= 0 && q1 >= q0 && int64_t(q1) <= p.Tq && k0 >= 0 && k1 >= k0 && int64_t(k1) <= p.Tk;
    nq = ok ? q1 - q0 : 0;
    nk = ok ? k1 - k0 : 0;
    return ok;
}

// Key blocks that the tile of `tt` tokens from token t0 of a sequence covers.
__device__ __forceinline__ int tile_blocks(int t0, int tt, int nq, int nk)
{
    const int64_t seen = int64_t(min(int64_t(nq), int64_t(t0) + tt)) + nk - nq;
    return seen <= 0 ? 0 : int((seen + kKeys - 1) / kKeys);
}

// Length of a tile on the work line: its blocks (one where there are none) and
// `extra` for what a tile costs besides (queries, epilogue).
__device__ __forceinline__ int tile_units(int blocks, int extra) { return max(1, blocks) + extra; }

// The block at unit x of a tile: the extra units come first.  A CTA whose
// share lies inside a tile has 1 + extra units of it or more (the shares are
// never shorter where extra > 0), so it has a block.
__device__ __forceinline__ int unit_block(int64_t x, int blocks, int extra)
{
    return int(max(int64_t(0), min(int64_t(blocks), x - extra)));
}

// sum_{i < x} floor(i / 2^k)
__device__ __forceinline__ int64_t shift_sum(int64_t x, int k)
{
    const int64_t q = x >> k;
    return ((q * (q - 1) / 2) << k) + q * (x - (q << k));
}

// sum_{i < n} floor((a i + b) / 128), a, b >= 0.  Multiples of 128 go to the
// sum directly.  What is left of a, if a power of two, makes a sum of shifts;
// else its terms step over at most a n / 128 multiples, and counting the i
// behind each of them is the same sum with a and 128 swapped.
__device__ __forceinline__ int64_t floor_sum128(int64_t n, int64_t a, int64_t b)
{
    int64_t sum = (a >> 7) * (n * (n - 1) / 2) + (b >> 7) * n;
    a &= 127;
    b &= 127;
    if ((a & (a - 1)) == 0) {
        const int k = a ? __ffs(int(a)) - 1 : 0;
        return a ? sum + shift_sum(n + (b >> k), 7 - k) - shift_sum(b >> k, 7 - k) : sum;
    }
    for (int64_t m = 128; a * n + b >= m;) {
        const int64_t top = a * n + b, t = m;
        n = top / m;
        b = top % m;
        m = a;
        a = t;
        sum += (a / m) * (n * (n - 1) / 2) + (b / m) * n;
        a %= m;
        b %= m;
    }
    return sum;
}

// Units, without extra ones, of the `tiles` tiles of a head of a sequence.
__device__ __forceinline__ int64_t head_units(int tt, int tiles, int nq, int nk)
{
    if (tiles == 0)
        return 0;
    const int64_t last = max(1, (nk + kKeys - 1) / kKeys);     // the last tile sees all keys
    if (tiles == 1)
        return last;
    // tile i before it ends with the keys below base + (i + 1) tt: the first
    // `blind` see none
    const int64_t base = int64_t(nk) - nq;
    const int64_t blind = base >= 0 ? 0 : min(tiles - 1, int(-base) / tt);
    return blind + floor_sum128(tiles - 1 - blind, tt, base + (blind + 1) * tt + 127) + last;
}

// ---------------------------------------------------------------- kernel

// mbar_wait of a whole warp.  All lanes try: with lane 0 alone (a predicated
// try and a vote) an 8192-token prompt took 427 us instead of 357, with a
// suspend-time hint 605.  Without a call: a kernel that moves registers between
// its warps (setmaxnreg) cannot hold one, since a callee's registers are not
// bounded.
__device__ __forceinline__ bool try_wait_warp(uint32_t bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
}

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *status,
                                          uint64_t limit_ns = kWaitLimitNs)
{
    if (!try_wait_warp(bar, parity)) {
        // the clock and the flag are read once in 64 tries: they would delay
        // the next try, and most waits are part of a chain of hand-offs
        uint64_t t0 = 0;
#pragma unroll 1
        for (uint32_t tries = 1; !try_wait_warp(bar, parity); ++tries) {
            if (tries % 64)
                continue;
            const uint64_t t = __shfl_sync(0xffffffffu, global_timer_ns(), 0);
            if (!t0)
                t0 = t;
            if (__any_sync(0xffffffffu, abort_flag && *abort_flag))
                return false;
            if (t - t0 > limit_ns) {
                if (abort_flag)
                    *abort_flag = 1;
                atomicExch(status, BL_ERR_TIMEOUT);
                return false;
            }
        }
    }
    return true;
}

constexpr uint64_t kDrainLimitNs = 100000000ull;

// A warp's wait; false if it was given up (the same for every lane).
#define BL_WAIT(bar, parity) wait_warp(smem_u32(&(bar)), (parity), abort_flag, p.status)

template <bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap, const PrefillParams p)
{
    constexpr int kStages = kv_stages<PAIR>();
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    Smem<PAIR> &sm = *reinterpret_cast<Smem<PAIR> *>(smem_raw);
    // the swizzled tiles begin at multiples of 1024 bytes, as declared (there
    // is no room to align by hand)
    if (smem_u32(smem_raw) & 1023u) {
        if (threadIdx.x == 0)
            atomicExch(p.status, BL_ERR_UNSUPPORTED);
        return;
    }
    volatile int *abort_flag = &sm.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&sm.kv_full[s]), 1);
            mbar_init(smem_u32(&sm.kv_empty[s]), 1);
            mbar_init(smem_u32(&sm.v_posted[s]), 1);
            mbar_init(smem_u32(&sm.v_fixed[s]), 32);
        }
        mbar_init(smem_u32(&sm.q_full), 1);
        mbar_init(smem_u32(&sm.q_empty), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&sm.s_full[s]), 1);
            mbar_init(smem_u32(&sm.p_full[s]), 4);          // a lane of each softmax warp
            mbar_init(smem_u32(&sm.o_full[s]), 1);
        }
        mbar_init(smem_u32(&sm.ml_full), 128);
        mbar_init(smem_u32(&sm.o1_read), 128);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(smem_u32(&sm.item_full[i]), 1);
            mbar_init(smem_u32(&sm.item_empty[i]), 10);     // a lane of each of the other warps
        }
        mbar_init(smem_u32(&sm.drain), 1);
        sm.abort_flag = 0;
        sm.poison_piece = -1;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kLoadWarp && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&qmap)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
    }
    if (warp == kMmaWarp)
        tmem_alloc(smem_u32(&sm.tmem_base), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp >= kLoadWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kLoadWarp) {
            // ---------------------------------------- work list, TMA loads
            const int TT = PAIR ? 2 * p.TM : p.TM;        // tokens of a tile
            // lane l holds sequence chunk + l
            int chunk = 0, l_q0 = 0, l_nq = 0, l_k0 = 0, l_nk = 0;
            auto load_chunk = [&](int b0) {
                chunk = b0;
                l_nq = l_nk = 0;
                return b0 + lane >= p.batch || sequence(p, b0 + lane, l_q0, l_nq, l_k0, l_nk);
            };
            // Two passes over the sequences, the first for the line's length:
            // it holds sums of blocks and of tiles apart, since the cost of a
            // tile beyond its blocks counts only where the shares are long.
            // The code runs once, from a cold instruction cache, so it is kept
            // small: no 64-bit division on the usual path.
            int64_t W = 0, w = 0, w_end = 0, off = 0, c = blockIdx.x, G = 0;
            int extra = 0, b = 0, q0 = 0, nq = 0, k0 = 0, nk = 0, kvh = 0, t0 = 0;
            // floor(a / W) and floor(a / G)
            auto over = [](int64_t a, int64_t d) {
                return (uint64_t(a) | uint64_t(d)) >> 32 ? a / d : int64_t(uint32_t(a) / uint32_t(d));
            };
            auto take_sequence = [&](int next) {
                b = next;
                if (b < chunk || b >= chunk + 32)
                    load_chunk(b & ~31);
                q0 = __shfl_sync(0xffffffffu, l_q0, b - chunk);
                nq = __shfl_sync(0xffffffffu, l_nq, b - chunk);
                k0 = __shfl_sync(0xffffffffu, l_k0, b - chunk);
                nk = __shfl_sync(0xffffffffu, l_nk, b - chunk);
            };
            bool fine = load_chunk(0);
            int64_t u = 0, incl = 0;     // units without extra ones of a head of lane's sequence; of the chunk's up to it
            int t = 0, tin = 0;          // the same of tiles
            for (int pass = 0; pass < 2; ++pass) {
                int64_t before = 0, tiles = 0;
                for (int b0 = 0; b0 < p.batch; b0 += 32) {
                    if (b0 != chunk)
                        fine = load_chunk(b0) && fine;
                    if (pass == 0 || p.batch > 32) {
                        t = tin = (l_nq + TT - 1) / TT;
                        u = incl = head_units(TT, t, l_nq, l_nk);
                        if (p.batch > 1) {
#pragma unroll
                            for (int o = 1; o < 32; o <<= 1) {
                                const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
                                const int z = __shfl_up_sync(0xffffffffu, tin, o);
                                incl += lane >= o ? v : 0;
                                tin += lane >= o ? z : 0;
                            }
                        }
                    }
                    if (pass) {
                        const int64_t upto = before + incl + int64_t(extra) * tin;
                        const unsigned past = __ballot_sync(0xffffffffu, upto * p.Hkv > w);
                        if (past) {
                            const int l = __ffs(past) - 1;
                            const int64_t per_head = __shfl_sync(0xffffffffu, u + int64_t(extra) * t, l);
                            off = w - (__shfl_sync(0xffffffffu, upto, l) - per_head) * p.Hkv;
                            take_sequence(b0 + l);
                            for (; off >= per_head; off -= per_head)
                                ++kvh;
                            break;
                        }
                    }
                    const int end = p.batch > 1 ? 31 : 0;
                    before += __shfl_sync(0xffffffffu, incl + int64_t(extra) * tin, end);
                    tiles += __shfl_sync(0xffffffffu, tin, end);
                }
                if (pass == 0) {
                    W = before * p.Hkv;
                    if (W >= 8 * int64_t(gridDim.x)) {
                        extra = kTileExtra;
                        W += extra * tiles * p.Hkv;
                    }
                    G = min(int64_t(gridDim.x), W);
                    if (c < G) {
                        w = over(c * W, G);
                        w_end = over((c + 1) * W, G);
                    }
                    if (w == w_end)
                        break;
                }
            }
            if (!fine && blockIdx.x == 0)
                atomicExch(p.status, BL_ERR_SHAPE);
            // the head's tile that holds unit off, 32 tiles at a time
            while (w < w_end && nq > TT) {
                const int64_t ti = int64_t(t0) + int64_t(lane) * TT;
                const int64_t len = ti < nq ? tile_units(tile_blocks(int(ti), TT, nq, nk), extra) : 0;
                int64_t upto = len;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
                    upto += lane >= o ? v : 0;
                }
                const unsigned past = __ballot_sync(0xffffffffu, upto > off);
                if (past) {
                    const int l = __ffs(past) - 1;
                    off -= __shfl_sync(0xffffffffu, upto - len, l);
                    t0 += l * TT;
                    break;
                }
                off -= __shfl_sync(0xffffffffu, upto, 31);
                t0 += 32 * TT;
            }
            if (lane == 0)
                p.hdr[c].valid = 0;
            int it = 0, loads = 0;       // pieces listed, blocks loaded
            int q_loads = 0;
            bool ok = true;
            auto load_q = [&](const Item &item) {
                if (!BL_WAIT(sm.q_empty, (uint32_t(q_loads) & 1u) ^ 1u))
                    return false;
                ++q_loads;
                const int qt = PAIR && item.toks > p.TM ? 2 : 1;
                if (lane == 0) {
                    const uint32_t bar = smem_u32(&sm.q_full);
                    mbar_arrive_tx(bar, uint32_t(qt * p.TM * p.G) * 256u);
                    for (int s = 0; s < qt; ++s) {
                        const uint32_t dst = smem_u32(sm.q[s]);
                        tma_load_4d(dst, &qmap, bar, 0, item.kvh * p.G, item.q_row + s * p.TM, 0);
                        tma_load_4d(dst + kBox, &qmap, bar, 0, item.kvh * p.G, item.q_row + s * p.TM, 1);
                    }
                }
                __syncwarp();
                return true;
            };
            for (; ok; ++it) {
                // the next piece with work: blocks, or a tile without keys (its rows get zeros)
                Item item = {};
                while (w < w_end && !item.valid) {
                    const int blocks = tile_blocks(t0, TT, nq, nk), units = tile_units(blocks, extra);
                    const int64_t take = min(units - off, w_end - w);
                    const int j0 = unit_block(off, blocks, extra), j1 = unit_block(off + take, blocks, extra);
                    if (j1 > j0 || (blocks == 0 && off == 0)) {
                        item.valid = 1;
                        item.kvh = kvh;
                        item.q_row = q0 + t0;
                        item.toks = min(TT, nq - t0);
                        item.lim0 = int(max(int64_t(-0x40000000), int64_t(t0) + 1 + nk - nq));
                        item.nk = nk;
                        item.k_row = k0;
                        item.j0 = j0;
                        item.n = j1 - j0;
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            if (PAIR) {
                                const int rows = min(item.toks - s * p.TM, p.TM);
                                const int kb = rows <= 0 ? 0 : tile_blocks(t0 + s * p.TM, rows, nq, nk);
                                item.nb[s] = max(0, min(j1, kb) - j0);
                            } else {
                                item.nb[s] = (item.n + 1 - s) / 2;
                            }
                        }
                        const bool begins = j0 == 0;
                        item.slot = begins && j1 == blocks ? -1 : begins ? 2 * int(c) + 1 : 2 * int(c);
                        if (begins && j1 < blocks && lane == 0) {
                            // the CTA that holds the tile's last unit
                            const int64_t last = over((w - off + units) * G + W - 1, W) - 1;
                            p.hdr[c] = JoinHeader{1, kvh, item.q_row, item.toks, int(last), {}};
                        }
                    }
                    w += take;
                    off += take;
                    if (off == units) {
                        off = 0;
                        t0 += TT;
                        if (t0 >= nq) {
                            t0 = 0;
                            if (++kvh == p.Hkv) {
                                kvh = 0;
                                if (w < w_end) {
                                    do
                                        take_sequence(b + 1);
                                    while (nq == 0);
                                }
                            }
                        }
                    }
                }
                const int islot = it % kItems;
                if (!BL_WAIT(sm.item_empty[islot], (uint32_t(it / kItems) & 1u) ^ 1u))
                    break;
                if (lane == 0) {
                    sm.item[islot] = item;
                    mbar_arrive(smem_u32(&sm.item_full[islot]));
                }
                __syncwarp();
                if (!item.valid)
                    break;
                if (item.n == 0)
                    continue;
                // The piece's blocks in the order in which the products take
                // them.  The first ones are asked for before the queries, whose
                // place is free only when every score product of the previous
                // piece is complete: their stages come free without these
                // queries, so the ring never waits for itself.
                const int n = item.n, masked = max(0, min(item.nk, item.lim0)) / kKeys - item.j0;
                // (the first piece's queries come first: their place is free)
                const int early = q_loads ? min(2 * n, kStages - 2) : 0;
                for (int x = 0; x < 2 * n && ok; ++x, ++loads) {
                    if (x == early)
                        ok = load_q(item);
                    bool is_v;
                    int i;
                    if (PAIR) {
                        is_v = x & 1;
                        i = x >> 1;
                    } else if (x < min(2, n)) {
                        is_v = false;
                        i = x;
                    } else {
                        // V(0), K(2), V(1), K(3), ..., V(n - 2), V(n - 1)
                        const int y = x - min(2, n);
                        is_v = !(y & 1) || y > 2 * (n - 2);
                        i = y > 2 * (n - 2) ? y - max(0, n - 2) : is_v ? y / 2 : y / 2 + 2;
                    }
                    const int st = loads % kStages;
                    ok = ok && (loads < kStages || BL_WAIT(sm.kv_empty[st], (uint32_t(loads / kStages) & 1u) ^ 1u));
                    if (!ok)
                        break;
                    if (lane == 0) {
                        const uint32_t bar = smem_u32(&sm.kv_full[st]), dst = smem_u32(sm.kv[st]);
                        const CUtensorMap *map = is_v ? &vmap : &kmap;
                        const int row = item.k_row + (item.j0 + i) * kKeys;
                        mbar_arrive_tx(bar, kTile);
                        tma_load_4d(dst, map, bar, 0, item.kvh, row, 0);
                        if (is_v && i >= masked)
                            mbar_arrive(smem_u32(&sm.v_posted[st]));
                    }
                    __syncwarp();
                }
                if (ok && early == 2 * n)       // all of them
                    ok = load_q(item);
            }
            // copies in flight have landed before the CTA exits (at once
            // unless another role gave up before it took them)
            for (int x = max(0, loads - kStages); x < loads; ++x)
                wait_warp(smem_u32(&sm.kv_full[x % kStages]), uint32_t(x / kStages) & 1u, nullptr, p.status,
                            kDrainLimitNs);
            if (q_loads)
                wait_warp(smem_u32(&sm.q_full), uint32_t(q_loads - 1) & 1u, nullptr, p.status, kDrainLimitNs);
        } else if (warp == kMmaWarp) {
            // ---------------------------------------- MMA issue
            const uint64_t q_desc = smem_desc_sw128(smem_u32(sm.q[0]));
            const uint64_t k_desc = smem_desc_sw128(smem_u32(sm.kv[0]));
            const uint64_t v_desc = smem_desc_mn_sw128(smem_u32(sm.kv[0]));
            int loads = 0, q_loads = 0;
            uint32_t fixed_parity = 0;              // bit per stage
            uint32_t p_parity[2] = {0, 0};
            bool ok = true, issued = false;
            // wait for load x
            auto landed = [&](int x) { return BL_WAIT(sm.kv_full[x % kStages], uint32_t(x / kStages) & 1u); };
            auto scores = [&](int s, int x) {
                tc_fence_after();
                mma_scores(tmem + uint32_t(s * kKeys), q_desc + uint64_t(PAIR ? s : 0) * (kTile >> 4),
                           k_desc + uint64_t(x % kStages) * (kTile >> 4));
                mma_commit(smem_u32(&sm.s_full[s]));
            };
            // O += P V of stream s (its weights are there); the products run in
            // the order of their issue, so the next scores may follow over P
            auto values = [&](int s, int x, bool first) {
                p_parity[s] ^= 1u;
                tc_fence_after();
                mma_values(tmem + uint32_t(256 + s * kHD), tmem + uint32_t(s * kKeys),
                           v_desc + uint64_t(x % kStages) * (kTile >> 4), first ? 0u : 1u);
            };
            // A check costs this warp 150 to 200 cycles even where the phase
            // is complete, and the tensor cores drain meanwhile, so the
            // barriers of one step are tried together: V of load xv, K of load
            // xk (-1: none) and the weights of stream s (-1: none).
            auto ready = [&](int xv, int xk, int s) {
                const uint32_t bv = smem_u32(&sm.kv_full[xv % kStages]), pv = uint32_t(xv / kStages) & 1u;
                const uint32_t bk = xk < 0 ? bv : smem_u32(&sm.kv_full[xk % kStages]);
                const uint32_t pk = xk < 0 ? pv : uint32_t(xk / kStages) & 1u;
                const uint32_t bp = s < 0 ? bv : smem_u32(&sm.p_full[s]);
                const uint32_t pp = s < 0 ? pv : s ? p_parity[1] : p_parity[0];
                const bool v = mbar_try_wait(bv, pv), k = mbar_try_wait(bk, pk), w = mbar_try_wait(bp, pp);
                if (__all_sync(0xffffffffu, v && k && w))
                    return true;
                return wait_warp(bv, pv, abort_flag, p.status) && wait_warp(bk, pk, abort_flag, p.status) &&
                       wait_warp(bp, pp, abort_flag, p.status);
            };
            for (int it = 0; ok; ++it) {
                const int islot = it % kItems;
                if (!BL_WAIT(sm.item_full[islot], uint32_t(it / kItems) & 1u))
                    break;
                const int valid = sm.item[islot].valid, n = sm.item[islot].n;
                const int nb0 = sm.item[islot].nb[0], nb1 = sm.item[islot].nb[1];
                const int masked = max(0, min(sm.item[islot].nk, sm.item[islot].lim0)) / kKeys - sm.item[islot].j0;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sm.item_empty[islot]));
                if (!valid)
                    break;
                if (n == 0)
                    continue;
                if (!BL_WAIT(sm.q_full, uint32_t(q_loads) & 1u))
                    break;
                ++q_loads;
                issued = true;      // from here on commits are in flight, which the drain below outlasts
                // non-finite values behind masks have been removed from V of block i, load x
                auto fixed = [&](int x, int i) {
                    if (i < masked)
                        return true;
                    const int st = x % kStages;
                    if (!BL_WAIT(sm.v_fixed[st], (fixed_parity >> st) & 1u))
                        return false;
                    fixed_parity ^= 1u << st;
                    return true;
                };
                auto release = [&](int x) { mma_commit(smem_u32(&sm.kv_empty[x % kStages])); };
                if (PAIR) {
                    if (!landed(loads))
                        break;
                    if (nb0)
                        scores(0, loads);
                    if (nb1)
                        scores(1, loads);
                    if (n == 1)
                        mma_commit(smem_u32(&sm.q_empty));
                    release(loads);
                    for (int i = 0; i < n; ++i) {
                        const int xv = loads + 2 * i + 1, xk = i + 1 < n ? xv + 1 : -1;
                        ok = ready(xv, xk, i < nb0 ? 0 : -1) && fixed(xv, i);
                        if (!ok)
                            break;
                        if (i < nb0) {
                            values(0, xv, i == 0);
                            if (i + 1 < nb0)
                                scores(0, xk);
                            else
                                mma_commit(smem_u32(&sm.o_full[0]));
                        }
                        if (i < nb1) {
                            ok = BL_WAIT(sm.p_full[1], p_parity[1]);
                            if (!ok)
                                break;
                            values(1, xv, i == 0);
                            if (i + 1 < nb1)
                                scores(1, xk);
                            else
                                mma_commit(smem_u32(&sm.o_full[1]));
                        }
                        release(xv);
                        if (xk >= 0)
                            release(xk);
                        if (i + 2 == n)
                            mma_commit(smem_u32(&sm.q_empty));
                    }
                } else {
                    for (int i = 0; i < min(2, n) && ok; ++i) {
                        ok = landed(loads + i);
                        if (ok) {
                            scores(i, loads + i);
                            if (i + 1 == n)
                                mma_commit(smem_u32(&sm.q_empty));
                            release(loads + i);
                        }
                    }
                    for (int i = 0; i < n && ok; ++i) {
                        // the next K is not waited for here: where memory sets the
                        // pace it arrives a block later
                        const int xv = loads + i + min(n, i + 2), s = i & 1;
                        ok = ready(xv, -1, s) && fixed(xv, i);
                        if (!ok)
                            break;
                        if (s)
                            values(1, xv, i < 2);
                        else
                            values(0, xv, i < 2);
                        release(xv);
                        if (i + 2 < n) {
                            ok = landed(xv + 1);
                            if (!ok)
                                break;
                            scores(s, xv + 1);
                            release(xv + 1);
                            if (i + 3 == n)
                                mma_commit(smem_u32(&sm.q_empty));
                        } else {
                            mma_commit(smem_u32(&sm.o_full[s]));
                        }
                    }
                }
                loads += 2 * n;
            }
            if (issued) {
                // every MMA has completed before tensor memory is released
                mma_commit(smem_u32(&sm.drain));
                wait_warp(smem_u32(&sm.drain), 0, nullptr, p.status, kDrainLimitNs);
            }
        } else if (warp == kFixWarp) {
            // ---------------------------------------- non-finite values behind masks
            int loads = 0;
            uint32_t posted_parity = 0;             // bit per stage
            bool ok = true;
            for (int it = 0; ok; ++it) {
                const int islot = it % kItems;
                if (!BL_WAIT(sm.item_full[islot], uint32_t(it / kItems) & 1u))
                    break;
                const int valid = sm.item[islot].valid, n = sm.item[islot].n, j0 = sm.item[islot].j0;
                const int nk = sm.item[islot].nk;
                const int full = max(0, min(nk, sm.item[islot].lim0)) / kKeys;
                for (int i = max(0, full - j0); i < n && ok && valid; ++i) {
                    const int x = loads + (PAIR ? 2 * i + 1 : i + min(n, i + 2)), st = x % kStages;
                    // this warp passes over the other blocks, so the stage's
                    // phase is the block's only once it has been asked for
                    ok = BL_WAIT(sm.v_posted[st], (posted_parity >> st) & 1u) &&
                         BL_WAIT(sm.kv_full[st], uint32_t(x / kStages) & 1u);
                    if (!ok)
                        break;
                    posted_parity ^= 1u << st;
                    // bf16 with all exponent bits set: exponent + 1 carries into the sign's place
                    uint4 *tile = reinterpret_cast<uint4 *>(sm.kv[st]);
                    uint32_t hit = 0;
#pragma unroll 8
                    for (int u = 0; u < int(kTile / 16) / 32; ++u) {
                        const uint4 v = tile[u * 32 + lane];
                        hit |= ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
                               ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
                    }
                    if (__any_sync(0xffffffffu, hit & 0x80008000u)) {
                        // rare: zero them, and note for each dimension the first
                        // key of the sequence whose value was not finite.  The
                        // notes of the previous piece have been read once both
                        // softmax groups have left it.
                        if (sm.poison_piece != it) {
                            if (it > 0 &&
                                !BL_WAIT(sm.item_empty[(it - 1) % kItems], uint32_t((it - 1) / kItems) & 1u)) {
                                ok = false;
                                break;
                            }
                            for (int d = lane; d < kHD; d += 32)
                                sm.poison[d] = 0x7fffffff;
                            __syncwarp();
                        }
                        for (int e = lane; e < int(kTile / 2); e += 32) {      // in memory order
                            unsigned short *q = reinterpret_cast<unsigned short *>(sm.kv[st]) + e;
                            if ((*q & 0x7f80u) == 0x7f80u) {
                                const int row = (e >> 6) & 127;                // key of the block
                                const int chunk = ((e >> 3) & 7) ^ (row & 7);  // the swizzle undone
                                const int d = (e >> 13) * 64 + chunk * 8 + (e & 7);
                                const int key = (j0 + i) * kKeys + row;
                                if (key < nk)
                                    atomicMin(&sm.poison[d], key);
                                *q = 0;
                            }
                        }
                        __syncwarp();
                        if (lane == 0)
                            sm.poison_piece = it;
                        __syncwarp();
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    }
                    mbar_arrive(smem_u32(&sm.v_fixed[st]));
                }
                loads += 2 * n;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sm.item_empty[islot]));
                if (!valid)
                    break;
            }
        }
    } else {
        // -------------------------------------------- softmax, one row per thread
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int s = warp >> 2;                            // stream
        const int r = threadIdx.x & 127;                    // row of the tile
        const uint32_t lanes = uint32_t(warp & 3) << 21;    // TMEM lanes 32 * (warp % 4) ..
        const uint32_t s_tmem = tmem + lanes + uint32_t(s * kKeys), o_tmem = tmem + lanes + uint32_t(256 + s * kHD);
        const int tok = r / p.G, g = r - tok * p.G;         // of the tile's rows
        uint32_t s_parity = 0, o_parity[2] = {0, 0}, ml_parity = 0, o1_parity = 0;
        bool o1_pending = false;                            // alt, stream 1: its last O may still be read
        for (int it = 0;; ++it) {
            const int islot = it % kItems;
            if (!BL_WAIT(sm.item_full[islot], uint32_t(it / kItems) & 1u))
                break;
            const Item &item = sm.item[islot];
            if (!item.valid)
                break;
            const int tt = (PAIR ? s * p.TM : 0) + tok;     // token of the tile
            const bool mine = tok < p.TM && tt < item.toks;
            const int limit = min(item.nk, item.lim0 + tt); // keys below are visible
            const int nb = item.nb[s];
            // blocks before this one are visible to every row of the stream
            const int full = max(0, min(item.nk, item.lim0 + (PAIR ? s * p.TM : 0))) / kKeys;
            float m = -INFINITY, l = 0.0f;
            bool ok = true;
            for (int i = 0; i < nb; ++i) {
                const int j = item.j0 + (PAIR ? i : 2 * i + s);
                if (!PAIR && i == 0 && o1_pending) {
                    // the product that the first weights release overwrites O
                    ok = BL_WAIT(sm.o1_read, o1_parity);
                    if (!ok)
                        break;
                    o1_parity ^= 1u;
                    o1_pending = false;
                }
                ok = BL_WAIT(sm.s_full[s], s_parity);
                if (!ok)
                    break;
                s_parity ^= 1u;
                tc_fence_after();
                uint32_t v[128];
                tmem_ld128_wait(s_tmem, v);
                if (j >= full) {
                    const int left = limit - j * kKeys;
#pragma unroll
                    for (int x = 0; x < 128; ++x)
                        v[x] = x < left ? v[x] : 0xff800000u;
                }
                float mx[4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    mx[x] = fmaxf(__uint_as_float(v[x]), __uint_as_float(v[x + 4]));
#pragma unroll
                for (int x = 8; x < 128; x += 8)
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        mx[y] = max3(mx[y], __uint_as_float(v[x + y]), __uint_as_float(v[x + y + 4]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if (i == 0) {
                    m = top;
                } else {
                    const bool grow = (top - m) * p.c > kRescale;
                    if (__any_sync(0xffffffffu, grow)) {
                        const float f = grow ? exp2_approx((m - top) * p.c) : 1.0f;
                        m = grow ? top : m;
                        l *= f;
                        // the scores' barrier covers every earlier product: O is idle
#pragma unroll 1
                        for (int x = 0; x < kHD; x += 32) {
                            uint32_t o[32];
                            tmem_ld32_wait(o_tmem + uint32_t(x), o);
#pragma unroll
                            for (int y = 0; y < 32; ++y)
                                o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                            tmem_st32_wait(o_tmem + uint32_t(x), o);
                        }
                    }
                }
                const float mc = m == -INFINITY ? 0.0f : m * p.c;
                l += row_weights(v, p.c, mc, s_tmem);
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sm.p_full[s]));
            }
            if (!ok)
                break;
            // ---- the piece's result: f0 * O of this stream (+ f1 * O of stream 1, alt)
            float f0 = 1.0f, f1 = 0.0f;
            bool second = false;
            if (!PAIR && s == 1) {
                if (nb) {
                    sm.ml[r] = make_float2(m, l);
                    mbar_arrive(smem_u32(&sm.ml_full));
                    o1_pending = true;
                }
            } else {
                if (nb) {
                    if (!BL_WAIT(sm.o_full[s], o_parity[0]))
                        break;
                    o_parity[0] ^= 1u;
                }
                if (!PAIR && item.nb[1]) {
                    if (!BL_WAIT(sm.ml_full, ml_parity) || !BL_WAIT(sm.o_full[1], o_parity[1]))
                        break;
                    ml_parity ^= 1u;
                    o_parity[1] ^= 1u;
                    second = true;
                    const float2 ml1 = sm.ml[r];
                    const float top = fmaxf(m, ml1.x);
                    f0 = m == -INFINITY ? 0.0f : exp2_approx((m - top) * p.c);
                    f1 = ml1.x == -INFINITY ? 0.0f : exp2_approx((ml1.x - top) * p.c);
                    l = l * f0 + ml1.y * f1;
                    m = top;
                }
                tc_fence_after();
                if (item.slot < 0) {
                    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                    f0 *= inv;
                    f1 *= inv;
                }
                const bool poisoned = *static_cast<volatile int *>(&sm.poison_piece) == it;
                __nv_bfloat16 *dst = p.out + int64_t(item.q_row + tt) * p.o_row + int64_t(item.kvh * p.G + g) * p.o_head;
                const bool aligned = reinterpret_cast<uintptr_t>(dst) % 32 == 0;
                const int64_t prow = int64_t(item.slot) * (PAIR ? 2 * kRows : kRows) + s * kRows + r;
                if (item.slot >= 0 && mine)
                    p.part_ml[prow] = make_float2(m, l);
                if (nb || item.slot < 0) {
#pragma unroll 1
                    for (int x = 0; x < kHD; x += 32) {
                        uint32_t o[32];
                        if (nb) {
                            tmem_ld32_wait(o_tmem + uint32_t(x), o);
                        } else {
#pragma unroll
                            for (int y = 0; y < 32; ++y)
                                o[y] = 0u;
                        }
                        float a[32];
#pragma unroll
                        for (int y = 0; y < 32; ++y)
                            a[y] = __uint_as_float(o[y]) * f0;
                        if (second) {
                            tmem_ld32_wait(o_tmem + uint32_t(kHD + x), o);
#pragma unroll
                            for (int y = 0; y < 32; ++y)
                                a[y] = fmaf(__uint_as_float(o[y]), f1, a[y]);
                        }
                        if (poisoned) {
#pragma unroll
                            for (int y = 0; y < 32; ++y)
                                if (limit > sm.poison[x + y])
                                    a[y] = __uint_as_float(0x7fffffffu);
                        }
                        if (!mine)
                            continue;
                        if (item.slot < 0) {
#pragma unroll
                            for (int y = 0; y < 32; y += 16) {
                                uint32_t w[8];
#pragma unroll
                                for (int z = 0; z < 8; ++z)
                                    w[z] = bf16x2(a[y + 2 * z], a[y + 2 * z + 1]);
                                store32(dst + x + y, w, aligned);
                            }
                        } else {
#pragma unroll
                            for (int y = 0; y < 32; y += 8) {
                                uint32_t w[8];
#pragma unroll
                                for (int z = 0; z < 8; ++z)
                                    w[z] = __float_as_uint(a[y + z]);
                                store32(p.part_o + prow * kHD + x + y, w, true);
                            }
                        }
                    }
                }
                if (!PAIR && second) {
                    tc_fence_before();
                    mbar_arrive(smem_u32(&sm.o1_read));
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&sm.item_empty[islot]));
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- joining the parts of cut tiles

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinSplit = 8;        // CTAs per cut tile, at most
constexpr int kJoinFew = 8;          // up to so many parts, a warp takes four rows at once,
constexpr int kJoinRows = 32;        // and where there are more rows than this
constexpr int kJoinLanes = 8;        // parts per lane: grids of up to 256 CTAs

// A part's share of the sum: 2^(c (m_part - m)) of its l and O.  A part in which
// the row sees no key has l = 0 and no O; NaN scores leave m at -inf and l NaN,
// and the factor is NaN then.
__device__ __forceinline__ float part_factor(float2 ml, float m, float c)
{
    return ml.y == 0.0f ? 0.0f : exp2f((ml.x - m) * c);
}

__device__ __forceinline__ void add_part(float4 &acc, float4 o, float f)
{
    if (f != 0.0f) {        // an O that was not written is not looked at
        acc.x = fmaf(o.x, f, acc.x);
        acc.y = fmaf(o.y, f, acc.y);
        acc.z = fmaf(o.z, f, acc.z);
        acc.w = fmaf(o.w, f, acc.w);
    }
}

// CTA (c, y) takes every gridDim.y-th group of rows of the tile whose first
// part CTA c of the main kernel holds.  The time is that of a few dependent
// loads, so many rows go side by side: four rows a warp, whose (m, l) come with
// one load and whose O's with independent ones; where few rows have many parts
// (single tokens on a long cache), the CTA's warps share a row's parts and add
// their sums in order.
template <bool PAIR>
__global__ void __launch_bounds__(kJoinThreads) prefill_join_kernel(const PrefillParams p)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float4 acc_s[kJoinWarps][32];
    __shared__ float fac_s[32 * kJoinLanes];
    const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint4 h0 = ld_dep_v4(&p.hdr[c]), h1 = ld_dep_v4(&p.hdr[c].last);
    if (!h0.x)
        return;
    const int kvh = int(h0.y), q_row = int(h0.z), toks = int(h0.w), parts = int(h1.x) - c + 1;
    constexpr int64_t kSlotRows = PAIR ? 2 * kRows : kRows;
    const int rows = toks * p.G;
    // row of part 0 in the workspace; part i: the first is the slot of a
    // tile's beginning, the others of a continuation
    auto slot_row = [&](int row) {
        const int tok = row / p.G, tile = PAIR ? tok / p.TM : 0;
        return tile * kRows + (tok - tile * p.TM) * p.G + (row - tok * p.G);
    };
    auto part_row = [&](int i, int at) { return int64_t(i ? 2 * (c + i) : 2 * c + 1) * kSlotRows + at; };
    auto load_ml = [&](int i, int at) { return __ldcg(&p.part_ml[part_row(i, at)]); };
    auto load_o = [&](int i, int at) {
        return __ldcg(reinterpret_cast<const float4 *>(p.part_o + part_row(i, at) * kHD) + lane);
    };
    auto store = [&](int row, const float4 &acc, float l) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int tok = row / p.G, g = row - tok * p.G;
        __nv_bfloat16 *dst = p.out + int64_t(q_row + tok) * p.o_row + int64_t(kvh * p.G + g) * p.o_head;
        *reinterpret_cast<uint2 *>(dst + 4 * lane) =
            make_uint2(bf16x2(acc.x * inv, acc.y * inv), bf16x2(acc.z * inv, acc.w * inv));
    };
    if (parts <= kJoinFew || rows > kJoinRows) {
        for (int row0 = (blockIdx.y * kJoinWarps + warp) * 4; row0 < rows; row0 += gridDim.y * kJoinWarps * 4) {
            // lane 8 r + i: row r, parts i, i + 8, ...
            const int mine = min(row0 + lane / 8, rows - 1), i = lane % 8, my_at = slot_row(mine);
            auto my_ml = [&](int j0) {
                return j0 + i < parts ? load_ml(j0 + i, my_at) : make_float2(-INFINITY, 0.0f);
            };
            const float2 first = my_ml(0);
            float m = first.x, l = 0.0f;
            for (int j0 = 8; j0 < parts; j0 += 8)
                m = fmaxf(m, my_ml(j0).x);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            float4 acc[4] = {};
            int at[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                at[r] = slot_row(min(row0 + r, rows - 1));
            for (int j0 = 0; j0 < parts; j0 += 8) {
                const float2 ml = j0 ? my_ml(j0) : first;
                const float f = part_factor(ml, m, p.c);
                l = fmaf(ml.y, f, l);
#pragma unroll 2
                for (int j = 0; j < min(8, parts - j0); ++j) {
                    float4 o[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        o[r] = load_o(j0 + j, at[r]);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        add_part(acc[r], o[r], __shfl_sync(0xffffffffu, f, 8 * r + j));
                }
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
                l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float lr = __shfl_sync(0xffffffffu, l, 8 * r);
                if (row0 + r < rows)
                    store(row0 + r, acc[r], lr);
            }
        }
        return;
    }
    for (int row = blockIdx.y; row < rows; row += gridDim.y) {
        const int at = slot_row(row);
        float2 ml[kJoinLanes];
        float m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int x = 0; x < kJoinLanes; ++x) {
            const int i = 32 * x + lane;
            ml[x] = i < parts ? load_ml(i, at) : make_float2(-INFINITY, 0.0f);
            m = fmaxf(m, ml[x].x);
        }
        m = warp_max(m);
#pragma unroll
        for (int x = 0; x < kJoinLanes; ++x) {
            const float f = part_factor(ml[x], m, p.c);
            l = fmaf(ml[x].y, f, l);
            if (warp == 0)
                fac_s[32 * x + lane] = f;
        }
        l = warp_sum(l);
        __syncthreads();
        float4 acc = {};
#pragma unroll 4
        for (int i = warp; i < parts; i += kJoinWarps) {
            const float f = fac_s[i];
            add_part(acc, f != 0.0f ? load_o(i, at) : make_float4(0.0f, 0.0f, 0.0f, 0.0f), f);
        }
        acc_s[warp][lane] = acc;
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int w = 1; w < kJoinWarps; ++w) {
                const float4 o = acc_s[w][lane];
                acc = make_float4(acc.x + o.x, acc.y + o.y, acc.z + o.z, acc.w + o.w);
            }
            store(row, acc, l);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- host side

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            ptr = nullptr;
        }
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

// [rows][heads][128] bf16 as a 4-D map of 64 values x heads x rows x 2 halves
// of the head: a box of both halves is the two swizzle-wide columns of an
// operand tile, one behind the other, in one copy.
int make_map(CUtensorMap *map, const bitlinear_heads &h, int heads, uint32_t box_heads, uint32_t box_rows,
             uint32_t box_halves)
{
    auto fn = encode_fn();
    if (!fn)
        return BL_ERR_CUDA;
    const cuuint64_t dims[4] = {kHD / 2, cuuint64_t(heads), cuuint64_t(h.rows), 2};
    const cuuint64_t strides[3] = {cuuint64_t(heads == 1 ? kHD : h.head_stride) * 2,
                                   cuuint64_t(h.rows == 1 ? kHD : h.row_stride) * 2, kHD};
    const cuuint32_t box[4] = {kHD / 2, box_heads, box_rows, box_halves}, estr[4] = {1, 1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, h.data, dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? BL_OK : BL_ERR_CUDA;
}

int main_grid(const DeviceInfo *di) { return std::min(di->sm_count, 32 * kJoinLanes); }

// Workspace: a join header per CTA, then the parts' m and l, then their O.
struct WsLayout {
    size_t ml, o, total;
};

WsLayout ws_layout(int grid)
{
    WsLayout w{};
    w.ml = (size_t(grid) * sizeof(JoinHeader) + 127) / 128 * 128;
    w.o = w.ml + size_t(grid) * 2 * (2 * kRows) * sizeof(float2);
    w.total = w.o + size_t(grid) * 2 * (2 * kRows) * kHD * sizeof(float) + 128;    // base rounded up
    return w;
}

template <bool PAIR>
int launch_mode(const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm, const PrefillParams &p, int grid,
                int64_t q_rows, int64_t k_rows, cudaStream_t s)
{
    int per_sm = 0;
    int st = occupancy(reinterpret_cast<const void *>(prefill_kernel<PAIR>), kThreads, smem_bytes<PAIR>(), &per_sm);
    if (st)
        return st;
    if (per_sm < 1)
        return BL_ERR_UNSUPPORTED;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<PAIR>();
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;       // each kernel waits itself for what came before it
    if ((st = cuda_status(cudaLaunchKernelEx(&cfg, prefill_kernel<PAIR>, qm, km, vm, p))))
        return st;
    // one block of keys at most for every tile: none is cut
    if (k_rows <= kKeys)
        return BL_OK;
    // rows of a tile that there can be, eight warps a CTA
    const int64_t rows = std::min<int64_t>(q_rows, (PAIR ? 2 : 1) * p.TM) * p.G;
    cfg.gridDim = dim3(unsigned(grid), unsigned(std::clamp<int64_t>(rows, 1, kJoinSplit)));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    return cuda_status(cudaLaunchKernelEx(&cfg, prefill_join_kernel<PAIR>, p));
}

}  // namespace

size_t attention_prefill_workspace_bytes(int, int)
{
    const DeviceInfo *di = device_info();
    return di ? ws_layout(main_grid(di)).total : 0;
}

int launch_attention_prefill(const PrefillArgs &a, cudaStream_t s)
{
    const DeviceInfo *di = device_info();
    if (!di)
        return BL_ERR_CUDA;
    const int grid = main_grid(di), G = a.H / a.Hkv;
    const WsLayout w = ws_layout(grid);
    auto *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(a.ws) + 127) / 128 * 128);
    PrefillParams p{};
    p.out = static_cast<__nv_bfloat16 *>(a.out.data);
    p.o_row = a.out.row_stride;
    p.o_head = a.out.head_stride;
    p.cu_q = a.cu_q;
    p.cu_k = a.cu_k;
    p.batch = a.batch;
    p.Hkv = a.Hkv;
    p.G = G;
    p.TM = kRows / G;
    p.Tq = a.q.rows;
    p.Tk = a.k.rows;
    p.c = a.scale * 1.44269504088896340736f;
    p.hdr = reinterpret_cast<JoinHeader *>(base);
    p.part_ml = reinterpret_cast<float2 *>(base + w.ml);
    p.part_o = reinterpret_cast<float *>(base + w.o);
    p.status = di->status;
    CUtensorMap qm, km, vm;
    int st;
    // (a tile of queries has TM * G rows, so its halves are copied apart)
    if ((st = make_map(&qm, a.q, a.H, uint32_t(G), uint32_t(p.TM), 1)) ||
        (st = make_map(&km, a.k, a.Hkv, 1, kKeys, 2)) || (st = make_map(&vm, a.v, a.Hkv, 1, kKeys, 2)))
        return st;
    // Pairs of tiles where there are as many as a quarter of the CTAs and the
    // sequences have 1 1/4 tiles or more (64 of 48 tokens on 500 others: pair
    // 54 us, alt 61; 64 of 32: 45 and 42; one of 2048: 43.2 and 44.9; 300 single
    // tokens on 1000: 176 and 149; one of 256 on 4000, 20 pairs: 32 and 28).
    const int64_t pairs = int64_t(a.Hkv) * (p.Tq / (2 * p.TM));
    return pairs >= grid / 4 && 4 * p.Tq >= 5 * int64_t(p.TM) * p.batch
               ? launch_mode<true>(qm, km, vm, p, grid, p.Tq, p.Tk, s)
               : launch_mode<false>(qm, km, vm, p, grid, p.Tq, p.Tk, s);
}

}  // namespace bl
