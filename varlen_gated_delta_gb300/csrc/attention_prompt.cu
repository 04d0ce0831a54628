// attention_prompt.cu - causal softmax attention of prompts and prompt slices on
// the tcgen05 tensor cores (bf16).
//
// For a tile of 128 queries, (token, head) pairs that share a key-value head, over tiles of BN keys:
//   S = Q K^T,  m' = max(m, rowmax S),  P = 2^(c (S - m')),  l' = l 2^(c (m - m')) + rowsum P,
//   O' = O 2^(c (m - m')) + P V,   c = scale log2(e),   out = O / l.
// 4 D operations for each visible (query, key): bound by the tensor cores, with
// the exponentials (one a score, on the special-function units) close behind.
//
// A CTA holds a pair of query tiles (one for D > 128) and every key tile it
// loads serves both.  Warp roles: one softmax warpgroup per query tile (a thread
// owns a row, so row maxima and sums need no exchange), one MMA warp per query
// tile, one TMA warp, one warp for the end of V.  S and O live in tensor memory;
// P replaces S in place as bf16 (A operand of the second product, read from
// tensor memory).  One tile's softmax runs under the other's products; with a
// single query tile S is double buffered instead and the scores of the next key
// tile run under the softmax.
//
// O is rescaled only when the row maximum has grown by more than 2^8 since the
// last time: P then stays below 2^8, with the same relative precision, and
// the division by l at the end uses the same reference.
//
// P = 0 for a masked score, and 0 * inf is NaN.  Rows of V past the end of the
// sequence (other sequences, stale cache slots) may hold anything: a warp zeroes
// them in shared memory before the product.  Masked tokens of the sequence itself
// are finite in sound data: when an output is not, the epilogue looks for a
// non-finite value among them, and where there is one the CTA takes its items a
// second time.  In that pass the warp also clears such values of the diagonal
// tiles, and the epilogue adds them to the rows that do see them.  8 x 4096 tokens, 32
// heads of 128 on 8, take 1910 us instead of 719 with one NaN near the end; 65536 tokens,
// 16 heads of 256 on 2, 61.0 ms instead of 30.1.
//
// A slice of a prompt over a long history has few items: its key tiles are then
// split, and each split leaves m, l and an unscaled o for a second kernel.
//
// Persistent CTAs, one per SM, take (query tile pair, head) items round by round
// in a fixed order, longest first by the tile's place in its sequence and to and
// fro over the CTAs; heads are innermost, so that the heads of a group read the
// same keys out of L2.
//
// 8 x 4096 tokens, 32 heads of 128 on 8: 806 us a call under sustained load, 1365 TFLOP/s
// of causal work, 0.70 of the measured bf16 burst rate and 0.78 of the sustained one (720
// us in a burst; the tensor pipe is active 0.69 of the cycles; what is left is the softmax
// between the products and each item's start and end).  16 x U[1, 4096] tokens, 16 heads
// of 64: 199 us, 754 TFLOP/s, bound by the softmax warpgroups, whose work a score is the
// same for half the products; no pipe of theirs is full (special functions 35%, issue
// slots 44%), they wait for tensor memory and for each other.  32 x U[1, 512], 32 heads on
// 8: 54 us, bound by the chain of one or two key tiles an item.
//
// Over a 4-bit cache (KV4) the load warp copies codes and scales to a ring of two tiles, and a fourth warpgroup turns them,
// and the queries, into fp16 tiles where the other instance's loads put bf16 ones.  4 x 512 tokens over 8192, 32 heads of
// 128 on 8: 231 us, 1150 TFLOP/s (tensor pipe 58% active); 256 items on 152 SMs leave a sixth of the time to the second
// round.  Steps: codes go to registers before the first is converted, which frees their place in the ring for the next copy,
// and a lane's places lie in different banks (286 -> 253 us); whole tiles take loads and stores at fixed offsets (253 -> 224).
// Loading codes into registers a tile ahead from global memory took 1393 (page lookups and divisions in the converting warps).
// 176 and 192 registers to a softmax thread instead of 184: 239 us against 224, and 275 against 253 a step earlier.  Taking the
// row's reference off the scores before the product with their factor costs 2 us, arrivals that follow from what was
// read (mbar_arrive_after) 5.
#include <algorithm>
#include <cmath>
#include <exception>
#include <map>
#include <mutex>
#include <utility>

#include "attention.cuh"
#include "kv4.cuh"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

// A try suspends the warp for up to 3.8 us: some 2 s of the kernel's own time, however long the GPU
// belongs to others meanwhile.
constexpr int kWaitTries = 1 << 19;
constexpr int kMaxBins = 4096;  // bins of the longest-first order (half for KV4, whose shared memory is full)
constexpr float kLazy = 8.f;    // growth of the row maximum (log2) that O waits for
constexpr float kKv4Shift = 7.f;  // log2 of the factor of fp16 probabilities: 2^(kLazy + 7) still fits

// Bounded waits of attention kernels that have given up.  It only grows, so that no query takes a report
// from another.
__device__ unsigned g_attention_timeouts;

// Registers a thread of this warpgroup gives up (Dec) or takes (Inc) from here on.
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// KV4: the cache holds 4-bit values (kv4.cuh).  The load warp copies codes and scales to a ring of their own, and a warpgroup
// more turns them, and the queries, into fp16 tiles.
template <int DP, bool KV4 = false>
struct Cfg {
    static constexpr int NQ = DP > 128 ? 1 : 2;    // query tiles of a CTA
    static constexpr int BN = DP > 128 ? 64 : 128; // keys of a tile
    static constexpr int NB = DP / 64;             // 64-channel blocks (128 swizzled bytes a row)
    static constexpr int QBYTES = 128 * DP * 2, SLOT = BN * DP * 2;
    static constexpr int SLOTS = 4;
    // Whether a softmax warpgroup passes its turn on after half of the exponentials: narrow heads
    // leave it more to do than the products (16 x 2048 tokens, 16 heads of 64: 200 -> 195 us; 8 x 4096,
    // 32 heads of 128: 729 -> 733).
    static constexpr bool EARLY = DP == 64;
    static constexpr int IO = KV4 ? 2 : 1;           // warpgroups beside the softmax ones
    static constexpr int THREADS = (NQ + IO) * 128;
    // registers a thread at launch and after the split: a softmax thread holds a row of scores
    static constexpr int REGS = 65536 / THREADS / 8 * 8 > 255 ? 248 : 65536 / THREADS / 8 * 8;
    static constexpr bool SPLIT_REGS = NQ == 2 || KV4;
    static constexpr int REGS_IO = !KV4 ? 96 : NQ == 2 ? 72 : 128;
    static constexpr int REGS_SOFTMAX = !SPLIT_REGS ? REGS : !KV4 ? 200 : NQ == 2 ? 184 : 248;
    static_assert(NQ * REGS_SOFTMAX + IO * REGS_IO <= (NQ + IO) * REGS, "more registers than the CTA was launched with");
    // KV4: codes and scales of a tile of keys (or values), and how many of those there are; inverse powers of the rows
    // of four items; the barriers of both, and which tokens of a raw tile are there
    static constexpr int RAW = BN * DP / 16 * 9, RAWS = 2;
    static constexpr int EXTRA = KV4 ? RAWS * RAW + 4 * 2 * 128 * 4 + 4 * 8 + RAWS * (2 * 8 + 8) : 0;
    static constexpr int MAX_BINS = KV4 ? kMaxBins / 2 : kMaxBins;
    // tensor memory: two score buffers, then O of each query tile
    static constexpr int COL_O = 2 * BN;
};

struct PromptParams {
    Attn a;
    int G;
    int tm;         // tokens of an item
    // What the two query tiles of an item hold, 128 rows each (one tile for D > 128):
    //   packed > 0: 2^packed heads of a group for each token, the second tile the next tokens;
    //   pair: 128 tokens of one head and of the next; neither: 256 tokens of one head.
    int packed, pair;
    int heads;      // items side by side
    int box_rows;   // key rows of a TMA box
    int bins, bin_shift;
    int min_rows;   // sequences with at most this many (query, head of a group) rows are not ours
    float c;        // |scale| log2(e)
    int negate;     // scale < 0
    int out32;      // output rows lie on 32-byte boundaries
    int splits;     // of the key tiles of an item; more than one: parts for a second kernel
    const float *ks;  // KV4: scales of the key heads, or NULL (the value heads' are a.out_scale)
    int q_wide;            // KV4: query rows lie on 16-byte boundaries
};

// Warp-wide mbarrier wait that gives up, for the whole warp, after so many tries or when another role has.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort, int tries = kWaitTries) {
    const uint32_t addr = smem_u32(bar);
    bool ok;
#pragma unroll 1
    while (!(ok = mbar_try_wait(addr, parity)) && !*abort)
        if (--tries < 0) {
            *abort = 1;
            atomicAdd(&g_attention_timeouts, 1u);
        }
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A warp's one arrival that frees what its lanes have read from shared memory; `read` holds bits of all that a lane has read.
// The lane that arrives follows from everybody's bits, so that the values have to be in registers before.  Behind a
// __syncwarp alone loads were seen to come after the arrival, when the next copy had begun to overwrite the place.
__device__ __forceinline__ void mbar_arrive_after(uint64_t *bar, uint32_t read) {
    const unsigned who = __ballot_sync(0xffffffffu, read & 1) & 31;
    if ((threadIdx.x & 31) == who) mbar_arrive(bar);
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int x,
                                            int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// D[tmem] (+)= A[tmem] B^T, issued by one thread.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Orders every use of loaded registers after the wait before it, for the compiler.
__device__ __forceinline__ void landed(uint32_t (&r)[32]) {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                     "+r"(r[i + 6]), "+r"(r[i + 7]));
}
// 32 bytes, to a 32-byte boundary.
__device__ __forceinline__ void store32(void *dst, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// True in one lane of the converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

constexpr int kMend = 1 << 16;  // marks the items of a second pass

// One item: tm tokens of sequence b from row0 on, of head h (with packing: of the heads of a group
// from h on), over its key tiles from lo on.
struct Item {
    int b, h, start, len, kv, row0;
    int split, lo;
    int n[2];     // key tiles of each query tile (0: no rows, or none that sees a key)
    int tiles;    // key tiles loaded
    int end;      // rows of the last key tile that hold keys; a second pass adds kMend
    // Keys from here on are hidden from the item's first row.
    __device__ __forceinline__ int masked() const { return kv - len + row0 + 1; }
    __device__ __forceinline__ uint32_t bits() const {
        return (uint32_t)(b ^ h ^ start ^ len ^ kv ^ row0 ^ split ^ lo ^ n[0] ^ n[1] ^ tiles ^ end);
    }
    // Whether V tile j has rows to change before they are used: past the last key, and in a second pass
    // those that are hidden from some row.
    __device__ __forceinline__ bool changes_v(int j, int BN) const {
        return (j + 1 == tiles && (end & (kMend - 1)) < BN) || (end >= kMend && (lo + j + 1) * BN > masked());
    }
};

template <int DP>
__device__ __forceinline__ int seq_tiles(const PromptParams &p, int b) {
    int start, len, kv;
    if (!attn_seq(p.a, b, start, len, kv) || (long)len * p.G <= p.min_rows) return 0;
    return (len + p.tm - 1) / p.tm;
}

// Tiles of a sequence of n tiles that fall into bin.
__device__ __forceinline__ int in_bin(int n, int bin, int shift) {
    return max(0, min(n - (bin << shift), 1 << shift));
}

// Warp-wide: item `idx`; false past the last one.  suffix[i]: tiles in bins >= i.
template <int DP>
__device__ __forceinline__ bool get_item(const PromptParams &p, const int *suffix, long idx, Item &it) {
    using C = Cfg<DP>;
    const int lane = threadIdx.x & 31;
    it.split = (int)(idx % p.splits);
    idx /= p.splits;
    if (idx >= (long)suffix[0] * p.heads) return false;
    int rank = (int)(idx / p.heads);
    it.h = (int)(idx % p.heads) << (p.packed + p.pair);
    int lo = 0, hi = p.bins - 1;  // the bin with suffix[bin + 1] <= rank < suffix[bin]
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (suffix[mid] > rank) lo = mid;
        else hi = mid - 1;
    }
    rank -= suffix[lo + 1];
    for (int b0 = 0; b0 < p.a.B; b0 += 32) {
        const int n = b0 + lane < p.a.B ? in_bin(seq_tiles<DP>(p, b0 + lane), lo, p.bin_shift) : 0;
        int sum = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += x;
        }
        const int all = __shfl_sync(0xffffffffu, sum, 31);
        if (rank >= all) {
            rank -= all;
            continue;
        }
        const int at = __ffs(__ballot_sync(0xffffffffu, rank < sum)) - 1;
        const int before = __shfl_sync(0xffffffffu, sum - n, at), mine = __shfl_sync(0xffffffffu, n, at);
        it.b = b0 + at;
        const int level = (lo << p.bin_shift) + mine - 1 - (rank - before);
        attn_seq(p.a, it.b, it.start, it.len, it.kv);
        it.row0 = level * p.tm;
        it.tiles = 0;
        const int shift = it.kv - it.len;
#pragma unroll
        for (int t = 0; t < C::NQ; ++t) {
            const int r = it.row0 + (p.pair ? 0 : t * (128 >> p.packed)), rows = min(128 >> p.packed, it.len - r);
            const int most = rows > 0 ? min(it.kv, shift + r + rows) : 0;
            it.n[t] = most > 0 ? (most + C::BN - 1) / C::BN : 0;
            it.tiles = max(it.tiles, it.n[t]);
        }
        it.end = min(C::BN, it.kv - (it.tiles - 1) * C::BN);
        it.lo = 0;
        if (p.splits > 1) {  // this split's key tiles
            const int per = (it.tiles + p.splits - 1) / p.splits, all = it.tiles;
            it.lo = min(it.split * per, all);
            it.tiles = min(all, it.lo + per) - it.lo;
            if (it.lo + it.tiles < all) it.end = C::BN;
#pragma unroll
            for (int t = 0; t < C::NQ; ++t) it.n[t] = max(0, min(it.n[t] - it.lo, it.tiles));
        }
        return true;
    }
    return false;
}

// Bits 0 and 1: the low and the high bf16 of x are not finite.
__device__ __forceinline__ uint32_t non_finite2(uint32_t x) {
    return ((x & 0x7f80u) == 0x7f80u ? 1u : 0u) | ((x & 0x7f800000u) == 0x7f800000u ? 2u : 0u);
}

// Warp-wide: non-finite values of the rows from `from` on of a V tile in shared memory become 0.
template <int DP>
__device__ __noinline__ void clear_non_finite(unsigned char *tile, int from) {
    for (int c = 0; c < Cfg<DP>::NB; ++c) {
        uint32_t *block = reinterpret_cast<uint32_t *>(tile + c * Cfg<DP>::BN * 128);
        for (int i = from * 32 + (threadIdx.x & 31); i < Cfg<DP>::BN * 32; i += 32) {
            const uint32_t x = block[i], which = non_finite2(x);
            if (which) block[i] = x & (which & 1u ? 0xffff0000u : 0xffffffffu) & (which & 2u ? 0x0000ffffu : 0xffffffffu);
        }
    }
}

// Warp-wide: whether V holds a non-finite value in channels c .. c + 31 of keys [k0, k1).  With `add`,
// each lane's row takes those of the keys before `seen` into its output (a part: into part).
__device__ __forceinline__ bool masked_non_finite(const PromptParams &p, int b, int start, int kvh, int c, int k0, int k1,
                                                  bool add, int seen, __nv_bfloat16 *out, float *part) {
    const int lane = threadIdx.x & 31, D = p.a.D;
    const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.a.v) + (long)kvh * D + c;
    const int words = min(32, D - c) / 8;  // of 16 bytes; none past the last channel
    float f[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = 0.f;
    bool found = false;
    for (int j0 = k0; j0 < k1; j0 += 32) {
        const long at = j0 + lane < k1 ? attn_key_row(p.a, b, start, j0 + lane, p.a.vs) : -1;
        uint32_t odd = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at >= 0 && i < words) {
                const uint4 x = __ldg(reinterpret_cast<const uint4 *>(v + at + i * 8));
                odd |= non_finite2(x.x) | non_finite2(x.y) | non_finite2(x.z) | non_finite2(x.w);
            }
        unsigned keys = __ballot_sync(0xffffffffu, odd != 0);
        found |= keys != 0;
        for (; add && keys != 0; keys &= keys - 1) {
            const int k = __ffs(keys) - 1;
            const long row = __shfl_sync(0xffffffffu, at, k);
            if (j0 + k >= seen) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < words) {
                    const uint4 x = __ldg(reinterpret_cast<const uint4 *>(v + row + i * 8));
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const uint32_t which = non_finite2(w[z]);
                        f[i * 8 + 2 * z] += which & 1u ? __uint_as_float(w[z] << 16) : 0.f;
                        f[i * 8 + 2 * z + 1] += which & 2u ? __uint_as_float(w[z] & 0xffff0000u) : 0.f;
                    }
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (f[i] != 0.f) {  // (NaN too)
            if (part) part[c + i] += f[i];
            else out[c + i] = __float2bfloat16_rn(__bfloat162float(out[c + i]) + f[i]);
        }
    return found;
}

// ---------------------------------------------------------------- the converting warpgroup (KV4)

// Rows of a query tile to fp16, each by the power of two that puts its largest value into [1, 2) (and the sign of the scale);
// the softmax factor of each row takes that back (its inverse).  tid: of the warpgroup.
template <int DP>
__device__ __forceinline__ void convert_queries(const PromptParams &p, const Item &it, int t, unsigned char *tile, float *inverses, int tid) {
    constexpr int LANES = DP / 8, STEP = 128 / LANES, BATCH = 4;  // lanes to a row, rows at a time, loads in flight
    const int c = tid % LANES;
#pragma unroll 1
    for (int r0 = tid / LANES; r0 < 128; r0 += STEP * BATCH) {
        Vec16<__nv_bfloat16> x[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int row = r0 + k * STEP;
            const int token = it.row0 + (p.pair ? 0 : t * (128 >> p.packed)) + (row >> p.packed);
            const int head = it.h + (p.pair ? t : row & ((1 << p.packed) - 1));
            x[k].u = make_uint4(0, 0, 0, 0);
            if (token < it.len && c * 8 < p.a.D) {
                const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(p.a.q) + (long)(it.start + token) * p.a.qs + (long)head * p.a.D + c * 8;
                if (p.q_wide) x[k].u = __ldg(reinterpret_cast<const uint4 *>(src));
                else
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[k].v[i] = src[i];
            }
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int row = r0 + k * STEP;
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(to_f32(x[k].v[i])));
#pragma unroll
            for (int d = LANES / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
            float back;
            const float power = kv4_row_power(amax, back) * (p.negate ? -1.f : 1.f);
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 h = __floats2half2_rn(to_f32(x[k].v[2 * i]) * power, to_f32(x[k].v[2 * i + 1]) * power);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
            *reinterpret_cast<uint4 *>(tile + (c >> 3) * 128 * 128 + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            if (c == 0) inverses[row] = back;
        }
    }
}

// A thread's part of a raw tile of keys (or values), 16 channels at a time.
template <int DP>
struct RawTile {
    static constexpr int BN = Cfg<DP, true>::BN, GROUPS = DP / 16, N = BN * GROUPS / 128;
    uint2 codes[N];
    uint32_t scale[N];
    // Bit i of `there`: tokens 16 i .. 16 i + 15 were copied; the others (past the last key, or of a page outside the cache)
    // read as zeros.
    __device__ __forceinline__ void load(int D, const unsigned char *raw, uint32_t there, int tid) {
        const int grp = tid % GROUPS, GR = D / 16, key0 = tid / GROUPS;
        if (there == (1u << (BN / 16)) - 1 && GR == GROUPS) {  // (as nearly all are)
            const unsigned char *at = raw + (key0 * GROUPS + grp) * 8, *s = raw + BN * GROUPS * 8 + key0 * GROUPS + grp;
#pragma unroll
            for (int i = 0; i < N; ++i) codes[i] = *reinterpret_cast<const uint2 *>(at + i * 1024), scale[i] = s[i * 128];
            return;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int key = key0 + i * (128 / GROUPS);
            codes[i] = make_uint2(0, 0), scale[i] = 0;
            if ((there >> (key >> 4) & 1) && grp < GR) {
                codes[i] = *reinterpret_cast<const uint2 *>(raw + (key * GR + grp) * 8);
                scale[i] = raw[BN * GR * 8 + key * GR + grp];
            }
        }
    }
    __device__ __forceinline__ uint32_t bits() const {
        uint32_t x = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) x ^= codes[i].x ^ codes[i].y ^ scale[i];
        return x;
    }
    // To fp16.  Groups of the upper 64 channels of 128 begin with their second half: 16 bytes of eight lanes then lie in different
    // banks.
    __device__ __forceinline__ void store(unsigned char *slot, int tid) const {
        const int grp = tid % GROUPS, turn = grp >> 2 & 1, key0 = tid / GROUPS;
        unsigned char *row = slot + (grp >> 2) * BN * 128 + key0 * 128;
        // (rows a multiple of eight apart swizzle alike)
        static_assert(128 / GROUPS % 8 == 0, "keys of a thread");
        unsigned char *at[2] = {row + ((((grp & 3) * 2 + turn) ^ (key0 & 7)) << 4), row + ((((grp & 3) * 2 + 1 - turn) ^ (key0 & 7)) << 4)};
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t s = kv4_scales(scale[i] | scale[i] << 8);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                uint32_t d[4];
                kv4_codes(z == turn ? codes[i].x : codes[i].y, d);
                *reinterpret_cast<uint4 *>(at[z] + i * (128 / GROUPS) * 128) =
                    make_uint4(mul_f16x2(d[0], s), mul_f16x2(d[1], s), mul_f16x2(d[2], s), mul_f16x2(d[3], s));
            }
        }
    }
};

template <int DP, bool KV4>
__global__ void __launch_bounds__(Cfg<DP, KV4>::THREADS, 1)
    attn_prompt_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const __grid_constant__ PromptParams p) {
    using C = Cfg<DP, KV4>;
    constexpr int NQ = C::NQ, BN = C::BN, NB = C::NB, SLOTS = C::SLOTS;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char *sq = smem, *ring = smem + NQ * C::QBYTES;
    unsigned char *raws = ring + SLOTS * C::SLOT;  // (this and the next three: KV4)
    float *inverses = reinterpret_cast<float *>(raws + C::RAWS * C::RAW);  // [4 items][2 query tiles][128 rows]
    uint64_t *f_full = reinterpret_cast<uint64_t *>(inverses + 4 * 2 * 128), *raw_full = f_full + 4, *raw_empty = raw_full + C::RAWS;
    volatile uint32_t *s_there = reinterpret_cast<uint32_t *>(raw_empty + C::RAWS);
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + SLOTS * C::SLOT + C::EXTRA);
    uint64_t *full = bars, *empty = full + SLOTS, *q_full = empty + SLOTS, *q_empty = q_full + 2,
             *s_full = q_empty + 2, *p_full = s_full + 2, *o_done = p_full + 2, *v_fixed = o_done + 2, *turn = v_fixed + SLOTS,
             *p_half = turn + 2, *item_full = p_half + 2, *item_empty = item_full + 4, *drained = item_empty + 4;
    Item *s_item = reinterpret_cast<Item *>(drained + 2);
    int *s_abort = reinterpret_cast<int *>(s_item + 4);
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(s_abort + 1);
    volatile int *s_again = s_abort + 2;
    int *suffix = s_abort + 4;  // [bins + 1]

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (the same in every lane, as the compiler sees it)
    // the last warpgroup: loads, products of each query tile, V values
    constexpr int kTmaWarp = NQ * 4, kMmaWarp = NQ * 4 + 1, kFixWarp = NQ * 4 + 3;

    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(full + i, KV4 ? 128 : 1);
            // every product warp and, for V (odd slots), the mending warp
            mbar_init(empty + i, KV4 ? NQ : NQ + (i & 1));
            mbar_init(v_fixed + i, 32);
            if (KV4) mbar_init(f_full + i, 128);
            if (KV4 && i < C::RAWS) mbar_init(raw_full + i, 1), mbar_init(raw_empty + i, 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + i, KV4 ? 128 : 1), mbar_init(q_empty + i, 1);
            mbar_init(s_full + i, 1), mbar_init(p_full + i, 128), mbar_init(o_done + i, 1);
            mbar_init(turn + i, 128), mbar_init(p_half + i, 128), mbar_init(drained + i, 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(item_full + i, 1), mbar_init(item_empty + i, NQ * 5 + (KV4 ? 4 : 1));
        fence_mbar_init();
        *s_abort = 0, *s_again = 0;
        if (!KV4) tma_prefetch_desc(&qmap), tma_prefetch_desc(&kmap), tma_prefetch_desc(&vmap);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(s_tmem, 512);
        tmem_relinquish();
    }
    pdl_wait_primary();
    // tiles per bin of places in a sequence, then suffix sums
    for (int i = tid; i <= p.bins; i += C::THREADS) suffix[i] = 0;
    __syncthreads();
    for (int b = tid; b < p.a.B; b += C::THREADS) {
        const int n = seq_tiles<DP>(p, b);
        for (int i = 0; (i << p.bin_shift) < n && i < p.bins; ++i) atomicAdd(suffix + i, in_bin(n, i, p.bin_shift));
    }
    __syncthreads();
    if (warp == 0) {
        int carry = 0;
        for (int i0 = (p.bins - 1) & ~31; i0 >= 0; i0 -= 32) {
            int x = i0 + lane < p.bins ? suffix[i0 + lane] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_down_sync(0xffffffffu, x, d);
                if (lane + d < 32) x += y;
            }
            x += carry;
            if (i0 + lane < p.bins) suffix[i0 + lane] = x;
            carry = __shfl_sync(0xffffffffu, x, 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    volatile int *abort = s_abort;
    Item it;
    it.n[1] = 0;
    // Items come from the load warp through a ring of four; false past the last one.
    uint32_t n_item = 0;
    auto next_item = [&](bool release = true) {
        const uint32_t k = n_item & 3;
        if (!wait_or_abort(item_full + k, (n_item >> 2) & 1, abort)) return false;
        it = s_item[k];
        __syncwarp();
        // (all lanes have read the same words)
        if ((release || it.b < 0) && lane == (int)(it.bits() & 31)) mbar_arrive(item_empty + k);
        ++n_item;
        return it.b >= 0;
    };

    if (warp >= kTmaWarp) {
        if constexpr (C::SPLIT_REGS) regs_dec<C::REGS_IO>();
        auto slot_of = [&](uint32_t s) { return s % SLOTS; };
        auto phase_of = [&](uint32_t s) { return (s / SLOTS) & 1; };
        uint32_t seq = 0;  // loads before this item: K_j is load seq + 2 j, V_j the one after it
        if (KV4 && warp >= kTmaWarp + 4) {
            // ------------------------------------------------------------ queries, keys and values to fp16
            if constexpr (KV4) {
                const int ctid = tid - (kTmaWarp + 4) * 32;
                uint32_t q_phase = 0;
                while (next_item()) {
                    const uint32_t k = (n_item - 1) & 3;
#pragma unroll 1
                    for (int t = 0; t < NQ; ++t) {
                        if ((t ? it.n[1] : it.n[0]) == 0) continue;
                        if (!wait_or_abort(q_empty + t, ((q_phase >> t) & 1) ^ 1, abort)) goto done;
                        q_phase ^= 1u << t;
                        convert_queries<DP>(p, it, t, sq + t * C::QBYTES, inverses + (k * 2 + t) * 128, ctid);
                        fence_async_smem();
                        mbar_arrive(q_full + t);
                    }
                    mbar_arrive(f_full + k);
#pragma unroll 1
                    for (int i = 0; i < 2 * it.tiles; ++i, ++seq) {
                        const uint32_t slot = slot_of(seq), r = seq % C::RAWS;
                        if (!wait_or_abort(raw_full + r, (seq / C::RAWS) & 1, abort)) goto done;
                        RawTile<DP> raw;
                        raw.load(p.a.D, raws + r * C::RAW, s_there[r], ctid);
                        mbar_arrive_after(raw_empty + r, raw.bits());
                        if (!wait_or_abort(empty + slot, phase_of(seq) ^ 1, abort)) goto done;
                        raw.store(ring + slot * C::SLOT, ctid);
                        fence_async_smem();
                        mbar_arrive(full + slot);
                    }
                }
            }
        } else if (warp == kTmaWarp) {
            // ------------------------------------------------------------ loads
            uint32_t q_phase = 0;
            const int boxes = BN / p.box_rows;  // boxes of a 64-channel block of a key tile
            // Every other round of items goes the other way round: the CTA that took the longest item
            // of one takes the shortest of the next.
            long first = 0;
            bool back = false, mending = false;
            auto send = [&]() {
                if (!wait_or_abort(item_empty + (n_item & 3), ((n_item >> 2) & 1) ^ 1, abort)) return false;
                if (lane == 0) {
                    s_item[n_item & 3] = it;
                    mbar_arrive(item_full + (n_item & 3));
                }
                ++n_item;
                return true;
            };
            while (true) {
                const bool more = get_item<DP>(p, suffix, first + (back ? gridDim.x - 1 - blockIdx.x : blockIdx.x), it);
                if (KV4) {
                    if (!more) it.b = -1;
                    if (!send()) goto done;
                    if (!more) break;
                    // pieces of box_rows tokens, that many to a tile; even lanes copy codes, odd ones scales
                    const int piece = lane >> 1, GR = p.a.D / 16, ps = p.a.page_size, kvh = it.h / p.G;
#pragma unroll 1
                    for (int j = 0; j < it.tiles; ++j) {
                        const int key = (it.lo + j) * BN + piece * p.box_rows, index = key / ps, at = key - index * ps;
                        int page = -1;
                        if (piece < boxes && key < it.kv) page = __ldg(p.a.block_table + (size_t)it.b * p.a.max_pages + index);
                        const bool read = page >= 0 && page < p.a.num_pages;
                        const uint32_t pieces = __ballot_sync(0xffffffffu, read && !(lane & 1));
                        uint32_t there = 0;  // blocks of 16 tokens of this piece, then of all
                        if (read) there = ((1u << (p.box_rows >> 4)) - 1u) << (piece * (p.box_rows >> 4));
                        there = __reduce_or_sync(0xffffffffu, there);
                        const long block = read ? ((long)page * p.a.HKV + kvh) * ((long)ps * GR * 9) : 0;
                        const long from = block + (lane & 1 ? ((long)ps * 8 + at) * GR : (long)at * GR * 8);
                        const uint32_t bytes = p.box_rows * GR * (lane & 1 ? 1 : 8), to = (lane & 1 ? BN * GR * 8 : 0) + piece * bytes;
#pragma unroll 1
                        for (int kv = 0; kv < 2; ++kv, ++seq) {
                            const uint32_t r = seq % C::RAWS;
                            if (!wait_or_abort(raw_empty + r, ((seq / C::RAWS) & 1) ^ 1, abort)) goto done;
                            if (lane == 0) {
                                s_there[r] = there;
                                mbar_arrive_expect_tx(raw_full + r, __popc(pieces) * p.box_rows * GR * 9);
                            }
                            __syncwarp();
                            if (read) bulk_load(raws + r * C::RAW + to, static_cast<const unsigned char *>(kv ? p.a.v : p.a.k) + from, bytes, raw_full + r);
                        }
                    }
                    first += gridDim.x, back = !back;
                    continue;
                }
                if (!more) {
                    // An item of nothing: when it has been taken, the items before it are at their end.  If one of
                    // them found cause, all are sent again.
                    it = Item{};
                    it.end = BN;
                    const uint32_t k = n_item & 3, phase = (n_item >> 2) & 1;
                    if (!mending && (!send() || !wait_or_abort(item_empty + k, phase, abort))) goto done;
                    if (!mending && *s_again) {
                        first = 0, back = false, mending = true;
                        continue;
                    }
                    it.b = -1;
                }
                if (mending) it.end += kMend;
                if (!send()) goto done;
                if (it.b < 0) break;
#pragma unroll
                for (int t = 0; t < NQ; ++t) {
                    if (it.n[t] == 0) continue;
                    if (!wait_or_abort(q_empty + t, ((q_phase >> t) & 1) ^ 1, abort)) goto done;
                    q_phase ^= 1u << t;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(q_full + t, C::QBYTES);
                        for (int c = 0; c < NB; ++c)
                            tma_load_3d(sq + t * C::QBYTES + c * 128 * 128, &qmap, q_full + t, c * 64,
                                        it.h + (p.pair ? t : 0),
                                        it.start + it.row0 + (p.pair ? 0 : t * (128 >> p.packed)));
                    }
                }
                for (int j = 0; j < it.tiles; ++j) {
                    // the row of this lane's box (packed keys: one box, at its token)
                    int row = it.start + (it.lo + j) * BN;
                    if (p.a.block_table != nullptr && lane < boxes) {
                        const int key = (it.lo + j) * BN + lane * p.box_rows;
                        const int page =
                            key < it.kv ? __ldg(p.a.block_table + (size_t)it.b * p.a.max_pages + key / p.a.page_size) : -1;
                        // outside the cache: past its end, where the load gives zeros
                        row = page < 0 || page >= p.a.num_pages ? p.a.num_pages * p.a.page_size
                                                                : page * p.a.page_size + key % p.a.page_size;
                    }
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t s = seq + 2 * j + kv, slot = slot_of(s);
                        if (!wait_or_abort(empty + slot, phase_of(s) ^ 1, abort)) goto done;
                        if (lane == 0) mbar_arrive_expect_tx(full + slot, C::SLOT);
                        __syncwarp();
                        if (lane < boxes) {
                            unsigned char *dst = ring + slot * C::SLOT + lane * p.box_rows * 128;
                            for (int c = 0; c < NB; ++c)
                                tma_load_3d(dst + c * BN * 128, kv ? &vmap : &kmap, full + slot, c * 64, it.h / p.G, row);
                        }
                    }
                }
                first += gridDim.x, back = !back, seq += 2 * it.tiles;
            }
        } else if (warp < kMmaWarp + NQ) {
            // ------------------------------------------------------------ products of query tile t
            const int t = warp - kMmaWarp;
            constexpr uint32_t kTypes = KV4 ? 1u << 7 | 1u << 10 : 0u;  // (without these bits: fp16)
            const uint32_t id_s = (idesc_bf16(128, BN, false, false) & ~kTypes) | (!KV4 && p.negate ? 1u << 13 : 0u);
            const uint32_t id_o = idesc_bf16(128, DP, false, true) & ~kTypes;
            const uint64_t qd0 = sdesc_sw128(smem_u32(sq) + t * C::QBYTES, 16, 1024);
            const uint32_t r_addr = smem_u32(ring), o_tmem = tmem + C::COL_O + t * DP;
            uint32_t q_phase = 0, p_phase = 0, fix_phase = 0;  // one bit a barrier
            for (; next_item(); seq += 2 * it.tiles) {
                const int n = NQ == 2 && t ? it.n[1] : it.n[0];
                auto wait_slot = [&](uint32_t s) { return wait_or_abort(full + slot_of(s), phase_of(s), abort); };
                // S[buf] = Q[t] K_j^T, and the slot is free after it
                auto scores = [&](int j) {
                    const int buf = NQ == 2 ? t : j & 1;
                    const uint32_t slot = slot_of(seq + 2 * j);
                    uint64_t kd = sdesc_sw128(r_addr + slot * C::SLOT, 16, 1024), qd = qd0;
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < DP / 16; ++ks)
                            mma_bf16(tmem + buf * BN, qd + (((ks >> 2) * 128 * 128 + (ks & 3) * 32) >> 4),
                                     kd + (((ks >> 2) * BN * 128 + (ks & 3) * 32) >> 4), id_s, ks > 0);
                        mma_commit(s_full + buf);
                        mma_commit(empty + slot);
                        if (j + 1 == n) mma_commit(q_empty + t);
                    }
                    __syncwarp();
                };
                if (n > 0) {
                    if (!wait_or_abort(q_full + t, q_phase, abort) || !wait_slot(seq)) goto done;
                    q_phase ^= 1;
                    tc_fence_after();
                    scores(0);
                }
                for (int j = 0; j < it.tiles; ++j) {
                    const uint32_t v = slot_of(seq + 2 * j + 1);
                    if (j >= n) {  // only the other query tile sees these keys: let the slots go by
                        if (!wait_slot(seq + 2 * j)) goto done;
                        if (elect_one()) mbar_arrive(empty + slot_of(seq + 2 * j));
                        __syncwarp();
                    } else if (j + 1 < n) {
                        if (!wait_slot(seq + 2 * j + 2)) goto done;
                        if (NQ == 1) tc_fence_after(), scores(j + 1);  // they run under this tile's softmax
                    }
                    // (all that the products wait for but P comes before P)
                    if (!wait_slot(seq + 2 * j + 1)) goto done;
                    if (!KV4 && it.changes_v(j, BN)) {
                        if (!wait_or_abort(v_fixed + v, (fix_phase >> v) & 1, abort)) goto done;
                        fix_phase ^= 1u << v;
                    }
                    if (j >= n) {
                        if (elect_one()) mbar_arrive(empty + v);
                        __syncwarp();
                        continue;
                    }
                    // O[t] (+)= P[buf] V_j
                    const int buf = NQ == 2 ? t : j & 1;
                    uint64_t vd = sdesc_sw128(r_addr + v * C::SLOT, BN * 128, 1024);
                    if (NQ == 2) {  // the first half of P is used while the second is computed
                        if (!wait_or_abort(p_half + buf, (p_phase >> buf) & 1, abort)) goto done;
                        tc_fence_after();
                        if (elect_one())
#pragma unroll
                            for (int ks = 0; ks < BN / 32; ++ks)
                                mma_bf16_ts(o_tmem, tmem + buf * BN + ks * 8, vd + ((ks * 2048) >> 4), id_o, j > 0 || ks > 0);
                        __syncwarp();
                    }
                    if (!wait_or_abort(p_full + buf, (p_phase >> buf) & 1, abort)) goto done;
                    p_phase ^= 1u << buf;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int ks = NQ == 2 ? BN / 32 : 0; ks < BN / 16; ++ks)
                            mma_bf16_ts(o_tmem, tmem + buf * BN + ks * 8, vd + ((ks * 2048) >> 4), id_o, j > 0 || ks > 0);
                        mma_commit(o_done + buf);
                        mma_commit(empty + v);
                    }
                    __syncwarp();
                    if (NQ == 2 && j + 1 < n) scores(j + 1);
                }
            }
        } else if (!KV4 && warp == kFixWarp) {
            // ------------------------------------------------------------ rows of V past the last key, and in
            // a second pass its non-finite values
            for (; next_item(); seq += 2 * it.tiles) {
                for (int j = 0; j < it.tiles; ++j) {
                    // every V tile is waited for, so that no phase of its barrier goes by unseen
                    const uint32_t s = seq + 2 * j + 1, slot = slot_of(s);
                    if (!wait_or_abort(full + slot, phase_of(s), abort)) goto done;
                    if (lane == 0) mbar_arrive(empty + slot);
                    if (!it.changes_v(j, BN)) continue;
                    unsigned char *tile = ring + slot * C::SLOT;
                    if (it.end >= kMend) clear_non_finite<DP>(tile, max(0, it.masked() - (it.lo + j) * BN));
                    if (j + 1 == it.tiles) {
                        const int end = it.end % kMend;
                        for (int c = 0; c < NB; ++c) {
                            uint4 *block = reinterpret_cast<uint4 *>(tile + c * BN * 128);
                            for (int i = end * 8 + lane; i < BN * 8; i += 32) block[i] = make_uint4(0, 0, 0, 0);
                        }
                    }
                    fence_async_smem();
                    mbar_arrive(v_fixed + slot);
                }
            }
        }
    } else {
        if constexpr (C::SPLIT_REGS) regs_inc<C::REGS_SOFTMAX>();
        // ---------------------------------------------------------------- softmax of query tile t
        const int t = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t o_col = lanes + C::COL_O + t * DP;
        uint32_t s_phase = 0, turn_phase = 0;
        uint32_t o_phase = 0;  // a bit for each score buffer: products with its P so far, mod 2
        if (NQ == 2 && t == 1) mbar_arrive(turn + 0);  // query tile 0 goes first
        while (next_item(!KV4)) {
            const int shift = it.kv - it.len, first = it.row0 + (p.pair ? 0 : t * (128 >> p.packed)),
                      r = first + (row >> p.packed);
            const int n = NQ == 2 && t ? it.n[1] : it.n[0];
            const int least = shift + first + 1;  // keys that the tile's first row sees
            float m = -INFINITY, l = 0.f;
            float pc = p.c;
            if constexpr (KV4) {
                const uint32_t k = (n_item - 1) & 3;
                if (!wait_or_abort(f_full + k, ((n_item - 1) >> 2) & 1, abort)) goto done;
                const float inverse = inverses[(k * 2 + t) * 128 + row];
                pc = n > 0 ? kv4_row_factor(p.c, inverse, p.ks ? __ldg(p.ks + it.h / p.G) : 1.f) : 1.f;
                // (not before: items without keys hold nobody up, and the inverses of the fourth item after this one may be
                // ready before a late warp has looked at these)
                mbar_arrive_after(item_empty + k, it.bits() ^ __float_as_uint(inverse) >> 23);
            }
            for (int j = 0; j < it.tiles; ++j) {
                if (j >= n) {  // only the other query tile sees these keys
                    if (!wait_or_abort(turn + t, turn_phase, abort)) goto done;
                    turn_phase ^= 1;
                    mbar_arrive(turn + 1 - t);
                    continue;
                }
                const int buf = NQ == 2 ? t : j & 1;
                if (!wait_or_abort(s_full + buf, (s_phase >> buf) & 1, abort)) goto done;
                s_phase ^= 1u << buf;
                if (NQ == 2) {
                    if (!wait_or_abort(turn + t, turn_phase, abort)) goto done;
                    turn_phase ^= 1;
                }
                tc_fence_after();
                const uint32_t s_col = lanes + buf * BN;
                uint32_t x[BN / 32][32];
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) tmem_ld32(s_col + c * 32, x[c]);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) landed(x[c]);
                if ((it.lo + j + 1) * BN > least) {  // some row does not see all of these keys
                    const int seen = shift + r + 1 - (it.lo + j) * BN;
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) {
                        // bit i: key c 32 + i is seen
                        const uint32_t bits = seen >= c * 32 + 32 ? 0xffffffffu : seen <= c * 32 ? 0u : (1u << (seen - c * 32)) - 1u;
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[c][i] = bits & (1u << i) ? x[c][i] : 0xff800000u;
                    }
                }
                float mx[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < BN / 32; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(x[c][i]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if (m == -INFINITY) m = top;  // nothing summed yet
                // rescale O when the reference of some row of the warp has to move
                const bool move = (top - m) * pc > kLazy;
                if (__any_sync(0xffffffffu, move)) {
                    const float f = move ? exp2_fast((m - top) * pc) : 1.f;
                    if (move) m = top, l *= f;
                    // (j > 0 here: a first tile sets m itself)
                    const int prev = NQ == 2 ? t : buf ^ 1;
                    if (!wait_or_abort(o_done + prev, ((o_phase >> prev) & 1) ^ 1, abort)) goto done;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < DP; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(o_col + c, o);
                        tmem_wait_ld();
                        landed(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st32(o_col + c, o);
                    }
                    tmem_wait_st();
                }
                // KV4 takes the reference off first: all exponents of a row share the rounding of m pc, and where that is large
                // (scores from 2^24 on) fp16 has no room for it
                const float mc = KV4 ? kKv4Shift : m == -INFINITY ? 0.f : -m * pc, base = m == -INFINITY ? 0.f : -m;
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int c = 0; c < BN / 64; ++c) {
                    uint32_t pk[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float2 s2 = make_float2(__uint_as_float(x[2 * c + (i >> 4)][(2 * i) & 31]),
                                                      __uint_as_float(x[2 * c + (i >> 4)][(2 * i + 1) & 31]));
                        float2 e = __ffma2_rn(KV4 ? __fadd2_rn(s2, make_float2(base, base)) : s2, make_float2(pc, pc),
                                              make_float2(mc, mc));
                        e.x = exp2_fast(e.x), e.y = exp2_fast(e.y);
                        sum = __fadd2_rn(sum, e);
                        if constexpr (KV4) {
                            const __half2 h = __floats2half2_rn(e.x, e.y);
                            pk[i] = *reinterpret_cast<const uint32_t *>(&h);
                        } else {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(e.x, e.y);
                            pk[i] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                    }
                    tmem_st32(s_col + c * 32, pk);
                    if (NQ == 2 && c == 0) {
                        tmem_wait_st();
                        tc_fence_before();
                        mbar_arrive(p_half + buf);
                        if (C::EARLY) mbar_arrive(turn + 1 - t);
                    }
                }
                if (NQ == 2 && !C::EARLY) mbar_arrive(turn + 1 - t);
                l += sum.x + sum.y;
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(p_full + buf);
                o_phase ^= 1u << buf;
            }
            // ---- out = O / l
            if (n > 0) {
                const int prev = NQ == 2 ? t : (n - 1) & 1;
                if (!wait_or_abort(o_done + prev, ((o_phase >> prev) & 1) ^ 1, abort)) goto done;
                tc_fence_after();
            }
            const bool whole = p.splits == 1;
            const float vs = KV4 && p.a.out_scale ? __ldg(p.a.out_scale + it.h / p.G) : 1.f;
            const float inv = !whole ? 1.f : l > 0.f ? 1.f / l : l;  // (0 gives 0, NaN stays)
            const int head = it.h + (p.pair ? t : row & ((1 << p.packed) - 1));
            const size_t out_row = (size_t)(it.start + r) * p.a.H + head;
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.a.out) + out_row * p.a.D;
            const Part part(p.a, p.splits, out_row, it.split);
            if (!whole && r < it.len) part.ml[0] = m * pc, part.ml[1] = l;
            uint32_t odd = 0;  // chunks of 32 channels with values that are not finite
            constexpr int OC = DP < 128 ? DP / 32 : 4;  // chunks loaded at a time
#pragma unroll 1
            for (int c0 = 0; c0 < DP; c0 += OC * 32) {
                __syncwarp();
                uint32_t o[OC][32];
                if (n > 0) {
#pragma unroll
                    for (int k = 0; k < OC; ++k) tmem_ld32(o_col + c0 + k * 32, o[k]);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < OC; ++k) landed(o[k]);
                } else {
#pragma unroll
                    for (int k = 0; k < OC; ++k)
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[k][i] = 0u;
                }
#pragma unroll
                for (int k = 0; k < OC; ++k) {
                    const int c = c0 + k * 32;
                    float2 finite[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};  // NaN when some value is not
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 f = __fmul2_rn(make_float2(__uint_as_float(o[k][2 * i]), __uint_as_float(o[k][2 * i + 1])),
                                                    make_float2(inv, inv));
                        if constexpr (KV4) f = __fmul2_rn(f, make_float2(vs, vs));
                        finite[i & 1] = __ffma2_rn(f, make_float2(0.f, 0.f), finite[i & 1]);
                        const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
                        w[i] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                    if (finite[0].x + finite[0].y + finite[1].x + finite[1].y != 0.f) odd |= 1u << (c >> 5);
                    if (r >= it.len) continue;
                    if (!whole) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            if (c + i < p.a.D) store32(part.o + c + i, &o[k][i]);
                    } else if (p.out32) {
                        if (c < p.a.D) store32(out + c, w);
                        if (c + 16 < p.a.D) store32(out + c + 16, w + 8);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (c + i * 8 < p.a.D)
                                *reinterpret_cast<uint4 *>(out + c + i * 8) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                    }
                }
            }
            __syncwarp();
            if (r >= it.len) odd = 0;
            // (a second pass: all keys that the V tiles were mended from)
            const bool mending = it.end >= kMend;
            const int k0 = max(it.lo * BN, mending ? it.masked() : least), k1 = min(it.kv, (it.lo + n) * BN);
            if (!KV4 && k0 < k1 && (mending || __any_sync(0xffffffffu, odd != 0))) {
                bool found = false;
#pragma unroll 1
                for (int c = 0; c < p.a.D; c += 32)
                    if (mending || __any_sync(0xffffffffu, (odd >> (c >> 5)) & 1))
                        found |= masked_non_finite(p, it.b, it.start, it.h / p.G, c, k0, k1, mending,
                                                   r < it.len ? min(it.kv, shift + r + 1) : 0, out, whole ? nullptr : part.o);
                if (!mending && found && lane == 0) {
                    *s_again = 1;
                    __threadfence_block();
                }
            }
            tc_fence_before();  // the next item's products follow this tile's next arrival
        }
    }
done:
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort) {  // copies and products in flight end before the CTA's memory goes
        if (KV4 && warp == kTmaWarp)
            for (int i = 0; i < C::RAWS; ++i) mbar_wait(raw_full + i, 0, 1000000), mbar_wait(raw_full + i, 1, 1000000);
        if (!KV4 && warp == kTmaWarp)
            for (int i = 0; i < SLOTS; ++i) {
                mbar_wait(full + i, 0, 1000000), mbar_wait(full + i, 1, 1000000);
                if (i < NQ) mbar_wait(q_full + i, 0, 1000000), mbar_wait(q_full + i, 1, 1000000);
            }
        if (warp >= kMmaWarp && warp < kMmaWarp + NQ) {
            if (elect_one()) mma_commit(drained + (warp - kMmaWarp));
            __syncwarp();
            mbar_wait(drained + (warp - kMmaWarp), 0, 10000000);
        }
        __syncthreads();
    }
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// A wait that nothing ends: how the way out of one is tested.
__global__ void wait_probe_kernel(int tries) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int s_abort;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
        s_abort = 0;
    }
    __syncwarp();
    wait_or_abort(&bar, 0, &s_abort, tries);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<EncodeTiledFn>(ptr);
    }();
    return fn;
}

// [rows][heads][D] bf16 with `stride` elements a row, read in boxes of 64 channels
// of box_heads heads and box_rows rows; channels past D and rows past the end read as 0.
bool encode_rows(CUtensorMap *map, const void *base, long rows, int heads, int D, long stride, int box_heads,
                 int box_rows) {
    const EncodeTiledFn enc = encode_fn();
    if (enc == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// log2 of the heads of a group that a query tile holds for each token: all of them, when they are a
// power of two and no sequence has the 128 tokens that would fill a tile with one head (slices of
// 64 tokens on 32768, 32 heads of 128 on 8: 81 us with one head a tile, 55 packed; long prompts are 4%
// slower packed, 8 x 4096 tokens: 719 and 749 us).
int packed_heads(int G, int max_q) {
    int n = 0;
    while (n < 7 && (G >> n) > 1) ++n;
    return G == 1 << n && max_q < 128 ? n : 0;
}
// Without that, two heads of a group are the two query tiles: they see the same keys to the same
// extent, and an item of 128 tokens leaves less of a short sequence unused than one of 256 (64 x 100
// tokens, 32 heads of 128 on 8: 70 us with 256 tokens, 53 with pairs).
bool paired_heads(int G, int D, int packed) { return packed == 0 && D <= 128 && G % 2 == 0; }

template <int DP, bool KV4>
cudaError_t launch(const Attn &a, int min_rows, int splits, cudaStream_t s, const float *ks = nullptr) {
    using C = Cfg<DP, KV4>;
    PromptParams p{};
    p.a = a;
    p.ks = ks;
    p.q_wide = rows_aligned(a.q, a.qs, a.D, 2);
    p.G = a.H / a.HKV;
    p.min_rows = min_rows;
    p.c = std::fmax(std::fabs(a.scale) * kLog2e, KV4 ? 0.f : 1e-30f);  // (KV4: kv4_row_factor)
    p.negate = a.scale < 0.f;
    p.out32 = ((uintptr_t)a.out & 31) == 0 && a.D % 16 == 0;
    const bool paged = a.block_table != nullptr;
    p.box_rows = C::BN;
    if (paged) while (a.page_size % p.box_rows != 0) p.box_rows /= 2;
    p.packed = packed_heads(p.G, a.max_q);
    p.pair = paired_heads(p.G, a.D, p.packed);
    p.tm = p.pair ? 128 : C::NQ * 128 >> p.packed;
    p.heads = a.H >> (p.packed + p.pair);
    const long levels = ((long)a.max_q + p.tm - 1) / p.tm;
    while (((levels + (1L << p.bin_shift) - 1) >> p.bin_shift) > C::MAX_BINS) ++p.bin_shift;
    p.bins = (int)((levels + (1L << p.bin_shift) - 1) >> p.bin_shift);
    const long kv_rows = paged ? (long)a.num_pages * a.page_size : a.N;
    CUtensorMap qm{}, km{}, vm{};
    if (!KV4 && (!encode_rows(&qm, a.q, a.N, a.H, a.D, a.qs, 1 << p.packed, 128 >> p.packed) ||
                 !encode_rows(&km, a.k, kv_rows, a.HKV, a.D, a.ks, 1, p.box_rows) ||
                 !encode_rows(&vm, a.v, kv_rows, a.HKV, a.D, a.vs, 1, p.box_rows)))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> attr_set{0};
    constexpr size_t kFixed = (size_t)C::NQ * C::QBYTES + C::SLOTS * C::SLOT + C::EXTRA + 512 + 1024;
    cudaError_t e = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(attn_prompt_kernel<DP, KV4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)(kFixed + (C::MAX_BINS + 1) * 4));
    });
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // at least four key tiles to a split
    const long key_tiles = paged ? ((long)a.max_pages * a.page_size + C::BN - 1) / C::BN : 1;
    p.splits = 1;
    while (p.splits * 2 <= splits && p.splits * 8 <= key_tiles) p.splits *= 2;
    const long items = ((long)a.N / p.tm + a.B) * p.heads * p.splits;
    const long grid = items < sms ? items : sms;
    e = launch_kernel(attn_prompt_kernel<DP, KV4>, dim3((unsigned)grid), dim3(C::THREADS), kFixed + (p.bins + 1) * 4, s,
                      true, qm, km, vm, p);
    note_launch();
    if (e != cudaSuccess || p.splits == 1) return e;
    return launch_attention_join(a, p.splits, min_rows, GDN_BF16, s);
}

// Splits of the key tiles when items are few: one request's slice of a prompt over a long history
// would keep a handful of CTAs busy (64 tokens on 32768, 32 heads of 128 on 8: 390 us, split 80).
// Sequences of at most min_rows (query, head of a group) rows have no items, and N tokens hold only so
// many longer ones.
int prompt_splits(int B, int N, int H, int HKV, int D, int max_q, int min_rows) {
    const int G = H / HKV, packed = packed_heads(G, max_q), pair = paired_heads(G, D, packed);
    const long seqs = std::min<long>(B, N / (min_rows / G + 1));
    const long tm = pair ? 128 : (D > 128 ? 128 : 256) >> packed, items = ((long)N / tm + seqs) * (H >> (packed + pair));
    int splits = 1;
    while (splits < 32 && items * splits * 2 <= 2 * 152) splits *= 2;
    return splits;
}

}  // namespace

size_t attention_prompt_part_floats(int B, int N, int H, int HKV, int D, int max_q) {
    const int splits = prompt_splits(B, N, H, HKV, D, max_q, kSplitRows);  // (fewer without that kernel)
    return splits == 1 ? 0 : (size_t)N * H * splits * (D + 2);
}

int attention_timeouts(cudaStream_t s, cudaError_t *e) {
    // What the last query on each stream has seen.
    static std::mutex lock;
    static std::map<std::pair<int, cudaStream_t>, unsigned> last;
    unsigned now = 0;
    int dev = 0;
    if ((*e = cudaGetDevice(&dev)) != cudaSuccess) return 0;
    *e = cudaMemcpyFromSymbolAsync(&now, g_attention_timeouts, sizeof(now), 0, cudaMemcpyDeviceToHost, s);
    if (*e == cudaSuccess) *e = cudaStreamSynchronize(s);
    if (*e != cudaSuccess) return 0;
    try {
        const std::lock_guard<std::mutex> hold(lock);
        unsigned &was = last[{dev, s}];
        const bool late = was != now;
        was = now;
        return late;
    } catch (const std::exception &) {  // (no memory: the next query tells)
        *e = cudaErrorMemoryAllocation;
        return 0;
    }
}

cudaError_t launch_attention_wait_probe(int tries, cudaStream_t s) {
    const cudaError_t e = launch_kernel(wait_probe_kernel, dim3(1), dim3(32), 0, s, false, tries);
    note_launch();
    return e;
}

bool attention_prompt_supported(const Attn &a, int dtype) {
    const bool paged = a.block_table != nullptr;
    return dtype == GDN_BF16 && rows_aligned(a.q, a.qs, a.D, 2) && rows_aligned(a.k, a.ks, a.D, 2) &&
           rows_aligned(a.v, a.vs, a.D, 2) && ((uintptr_t)a.out & 15) == 0 && (!paged || a.page_size % 8 == 0);
}

cudaError_t launch_attention_prompt(const Attn &a, int min_rows, cudaStream_t s) {
    const int splits = a.part == nullptr ? 1 : prompt_splits(a.B, a.N, a.H, a.HKV, a.D, a.max_q, min_rows);
    if (a.D <= 64) return launch<64, false>(a, min_rows, splits, s);
    if (a.D <= 128) return launch<128, false>(a, min_rows, splits, s);
    return launch<256, false>(a, min_rows, splits, s);
}

cudaError_t launch_attention_prompt_kv4(const Attn &a, const float *ks, int min_rows, cudaStream_t s) {
    const int splits = prompt_splits(a.B, a.N, a.H, a.HKV, a.D, a.max_q, min_rows);
    if (a.D <= 64) return launch<64, true>(a, min_rows, splits, s, ks);
    if (a.D <= 128) return launch<128, true>(a, min_rows, splits, s, ks);
    return launch<256, true>(a, min_rows, splits, s, ks);
}

}  // namespace gdn
