// attention_kv4.cu - gdn_attention_paged_kv4: attention of new tokens over a paged cache of 4-bit values (kv4.cuh).
//
// As gdn_attention_paged, with k_j = ks u_j c_j and v_j likewise; the heads' own scales ks and vs go into the softmax's
// factor and the output, so that what is multiplied, s c, is exact in fp16.  Queries are brought to the same type: each row by
// a power of two that puts its largest value into [1, 2), which the row's softmax factor takes back.  That keeps a bf16 query
// exact (down to 2^-24 of the row's largest value); an fp32 query is the sum of two fp16 values.  Probabilities
// are taken 2^14 times as large, so that fp16 holds them to 11 bits down to 2^-28 of the row's largest; with
// fp32 activations they too are sums of two.
//
// Keys are read once for the rows that share them, 9/16 bytes a channel of k and v: bound by HBM for few rows, by the
// tensor cores for many.  Three kernels, by a sequence's rows (tokens times the heads of a group):
// - up to 16 to 64 (see narrow_rows): blocks of 8 or 16 rows, values converted in the registers that a product reads (below);
// - more, bf16: the tcgen05 kernel of attention_prompt.cu, with a warpgroup that converts;
// - more, fp32: tiles of 64 rows by 64 keys, converted to fp16 in shared memory, 16-row mma.sync, products of both parts.
// The first and the last cut the work by key tiles: the tiles of all (sequence, row block, key-value head) triples form one
// list, of which every CTA takes an equal run; a CTA whose run begins or ends inside a triple leaves m, l and an
// unscaled o for a second kernel that joins the parts.  Which parts exist follows from the lengths alone.
//
// 64 requests with histories of U[1, 8192] tokens, one token each, 32 heads of 128 on 8: 68 us, 3.9 TB/s.  Longer ones add 55 us
// for 302 MB (5.5 TB/s, 0.81 of the measured copy), on top of some 15 us for launches, first dependent loads, the first tile
// and the join (one request: 16384 tokens 16 us, 131072 41, 524288 123).  What bounds the rest is issue and latency: 336
// instructions a warp for 16 keys of 128 channels, of which 128 convert and interleave, 64 scale and 16 multiply; 12 warps an SM
// issue 2.2 a clock.  Before the join took its present form (43 us for the request of 131072 tokens), 32 and 48 keys a warp at a
// time with 16 warps an SM gave 45 and 46 us, scoring two or four blocks of keys in turn 43 and 44.
#include <algorithm>
#include <cmath>

#include "attention.cuh"
#include "kv4.cuh"
#include "sm100.cuh"

namespace gdn {
namespace {

constexpr int kMaxSms = 160;
constexpr float kShift = 14.f;  // log2 of the probabilities' factor

struct Kv4Params {
    Attn a;
    const float *ks, *vs;  // of each key-value head, or NULL
    int G;
    float c;       // |scale| log2(e)
    float sign;    // of scale
    int blocks;    // row blocks of the longest sequence
    int page_shift;  // log2 of page_size, or -1
    int q_wide;      // query rows lie on 16-byte boundaries
    int min_rows, max_rows;  // sequences of more than min_rows and at most max_rows rows are ours
    int2 *spans;   // [B][blocks][HKV]: first and last CTA of a triple
    float *part;   // [2 * CTAs][ROWS * (3 + DP)]
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes to shared memory, or zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// What fp16 leaves of two values.
__device__ __forceinline__ uint32_t rest_f16(float lo, float hi, uint32_t kept) {
    const float2 f = f16x2_to_f32(kept);
    return pack_f16(lo - f.x, hi - f.y);
}
template <typename T>
__device__ __forceinline__ void store2(T *at, float x, float y);
template <>
__device__ __forceinline__ void store2(float *at, float x, float y) { *reinterpret_cast<float2 *>(at) = make_float2(x, y); }
template <>
__device__ __forceinline__ void store2(__nv_bfloat16 *at, float x, float y) {
    *reinterpret_cast<__nv_bfloat162 *>(at) = __floats2bfloat162_rn(x, y);
}
// Byte offset of 16-byte chunk c of row r: chunks of 8 neighbouring rows fall into different banks.
template <int DP>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return (uint32_t)(r * DP * 2 + ((c ^ (r & 7)) << 4));
}

// ---------------------------------------------------------------- the list of tiles

// The key tiles of one row block (ROWS rows) of sequence b, whose rows number len * G.
__device__ __forceinline__ int block_tiles(const Kv4Params &p, int rows, int keys, int block, int len, int kv) {
    const long last = min((long)(block + 1) * rows, (long)len * p.G) - 1;
    const int seen = min(kv, kv - len + (int)(last / p.G) + 1);
    return seen > 0 ? (seen + keys - 1) / keys : 1;  // (no keys: one tile that gives zeros)
}
// Row blocks of sequence b; 0: not ours.
__device__ __forceinline__ int seq_blocks(const Kv4Params &p, int rows, int b, int &start, int &len, int &kv) {
    if (b >= p.a.B || !attn_seq(p.a, b, start, len, kv)) return 0;
    if ((long)len * p.G <= p.min_rows || (long)len * p.G > p.max_rows) return 0;
    return (int)(((long)len * p.G + rows - 1) / rows);
}
// What beginning and ending a triple costs stands in the list as places before its first tile: without them a CTA with a
// run of short histories would take far longer than the others (64 x U[1, 8192] keys: 80 us without, 71 with one place, 72 with two;
// the join has since taken 3 us from each).
struct List {
    int rows, keys, ahead;  // rows of a block, keys of a tile, places before a triple's first tile
};
__device__ __forceinline__ long seq_places(const Kv4Params &p, List list, int b) {
    int start, len, kv;
    const int n = seq_blocks(p, list.rows, b, start, len, kv);
    long all = 0;
    for (int i = 0; i < n; ++i) all += list.ahead + block_tiles(p, list.rows, list.keys, i, len, kv);
    return all * p.a.HKV;
}

// A place in the list: tiles below 0 are those before a triple's first one.
struct Cursor {
    int b, block, h, tile, tiles, blocks, start, len, kv;
};
__device__ __forceinline__ void advance(const Kv4Params &p, List list, Cursor &x) {
    if (++x.tile < x.tiles) return;
    x.tile = -list.ahead;
    if (++x.h < p.a.HKV) return;
    x.h = 0;
    if (++x.block == x.blocks) {
        x.block = 0;
        do x.blocks = seq_blocks(p, list.rows, ++x.b, x.start, x.len, x.kv);
        while (x.blocks == 0 && x.b < p.a.B);
        if (x.blocks == 0) return;
    }
    x.tiles = block_tiles(p, list.rows, list.keys, x.block, x.len, x.kv);
}

// Block-wide: this CTA's run [u0, u1) of the U places and its first one; false when it has none.
template <int THREADS>
__device__ __forceinline__ bool find_run(const Kv4Params &p, List list, long long &u0, long long &u1, long long &U,
                                         long long &ctas, Cursor &cur) {
    __shared__ long long s_scan[THREADS / 32], s_at;
    __shared__ int s_b;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.a.B + THREADS - 1) / THREADS;  // threads own neighbouring sequences
    long long mine = 0;
    for (int i = 0; i < per; ++i) mine += seq_places(p, list, tid * per + i);
    long long sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += x;
    }
    if (lane == 31) s_scan[warp] = sum;
    __syncthreads();
    U = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) sum += s_scan[w];
        U += s_scan[w];
    }
    ctas = U < gridDim.x ? U : gridDim.x;  // every CTA that takes part has at least one place
    const long long cta = blockIdx.x;
    if (cta >= ctas) return false;
    u0 = cta * U / ctas, u1 = (cta + 1) * U / ctas;
    long long at = sum - mine;
    if (u0 >= at && u0 < sum)
        for (int i = 0; i < per; ++i) {
            const long long n = per > 1 ? seq_places(p, list, tid * per + i) : mine;
            if (u0 < at + n) {
                s_at = at, s_b = tid * per + i;
                break;
            }
            at += n;
        }
    __syncthreads();
    cur.b = s_b;
    cur.blocks = seq_blocks(p, list.rows, cur.b, cur.start, cur.len, cur.kv);
    long long left = u0 - s_at;
    for (cur.block = 0;; ++cur.block) {
        cur.tiles = block_tiles(p, list.rows, list.keys, cur.block, cur.len, cur.kv);
        if (left < (long long)(list.ahead + cur.tiles) * p.a.HKV) break;
        left -= (long long)(list.ahead + cur.tiles) * p.a.HKV;
    }
    cur.h = (int)(left / (list.ahead + cur.tiles));
    cur.tile = (int)(left % (list.ahead + cur.tiles)) - list.ahead;
    return true;
}

__device__ __forceinline__ long span_of(const Kv4Params &p, const Cursor &x) {
    return ((long)x.b * p.blocks + x.block) * p.a.HKV + x.h;
}
__device__ __forceinline__ float head_scale(const float *s, int h) { return s ? __ldg(s + h) : 1.f; }

// Block of 16 tokens of a cache: its page's (key-value head) block, or NULL.
__device__ __forceinline__ const uint8_t *token_block(const Kv4Params &p, const void *cache, int b, int h, int key) {
    const int page = __ldg(p.a.block_table + (size_t)b * p.a.max_pages + key / p.a.page_size);
    if (page < 0 || page >= p.a.num_pages) return nullptr;
    return static_cast<const uint8_t *>(cache) + ((long)page * p.a.HKV + h) * ((long)p.a.page_size * (p.a.D / 16) * 9);
}

// ---------------------------------------------------------------- rows by the block of 64 (fp32)

template <int DP, typename T>
struct Wide {
    static constexpr int KEYS = 64, ROWS = 64, THREADS = 128, STAGES = 3;
    static constexpr int Q = sizeof(T) == 4 ? 2 : 1;            // fp16 values to a query's
    static constexpr int RAW = KEYS * DP / 16 * 9;              // bytes of a tile of K (or V): codes, then scales
    static constexpr int TILE = KEYS * DP * 2;                  // the same in fp16
    static constexpr int QBYTES = ROWS * DP * 2;
    static constexpr int SMEM = STAGES * 2 * RAW + 2 * TILE + Q * QBYTES;
    static constexpr int PART = ROWS * (3 + DP);  // floats of a part: m, l, the rows' factors, o
    static constexpr int PER_SM = 220 * 1024 / (SMEM + 1024);
};

template <int DP, typename T>
__global__ void __launch_bounds__(128) kv4_wide_kernel(const Kv4Params p) {
    using C = Wide<DP, T>;
    constexpr int KEYS = C::KEYS, STAGES = C::STAGES;
    constexpr List kList = {C::ROWS, KEYS, 0};
    constexpr bool F32 = sizeof(T) == 4;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float s_c[C::ROWS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const uint32_t raw = sm100::smem_u32(smem), s_k = raw + STAGES * 2 * C::RAW, s_v = s_k + C::TILE, s_q = s_v + C::TILE;
    unsigned char *tiles = smem + STAGES * 2 * C::RAW, *q_rows = tiles + 2 * C::TILE;
    const int D = p.a.D, G = p.G, GR = D / 16;
    pdl_wait_primary();
    pdl_launch_dependents();  // (the joining blocks wait for this grid's end)
    long long u0, u1, U, ctas;
    Cursor cur;
    if (!find_run<C::THREADS>(p, kList, u0, u1, U, ctas, cur)) return;
    const long long cta = blockIdx.x;
    if (D < DP)  // channels past the last: zeros, for good
        for (int i = tid; i < 2 * KEYS * (DP / 8); i += C::THREADS)
            *reinterpret_cast<uint4 *>(tiles + (i / (KEYS * (DP / 8))) * C::TILE + chunk_at<DP>(i / (DP / 8) % KEYS, i % (DP / 8))) =
                make_uint4(0, 0, 0, 0);

    auto fetch = [&](const Cursor &x, int stage) {
        const uint32_t dst = raw + stage * 2 * C::RAW;
        const int codes = 8 * GR, per = 9 * GR;  // 16-byte chunks of 16 tokens
#pragma unroll 1
        for (int i = tid; i < KEYS / 16 * per; i += C::THREADS) {
            const int block = i / per, c = i % per, key = x.tile * KEYS + block * 16;
            const uint8_t *kb = nullptr, *vb = nullptr;
            if (key < x.kv) kb = token_block(p, p.a.k, x.b, x.h, key), vb = token_block(p, p.a.v, x.b, x.h, key);
            const int at = key % p.a.page_size;
            const long from = c < codes ? (long)at * GR * 8 + c * 16 : (long)p.a.page_size * GR * 8 + at * GR + (c - codes) * 16;
            const uint32_t to = c < codes ? block * codes * 16 + c * 16 : KEYS * GR * 8 + block * GR * 16 + (c - codes) * 16;
            copy16(dst + to, kb ? kb + from : p.a.k, kb != nullptr);
            copy16(dst + C::RAW + to, vb ? vb + from : p.a.v, vb != nullptr);
        }
    };
    Cursor ahead = cur;
    long long u_ahead = u0;
    for (int i = 0; i < STAGES - 1; ++i) {
        if (u_ahead < u1) {
            fetch(ahead, i);
            if (++u_ahead < u1) advance(p, kList, ahead);
        }
        copy_commit();
    }

    float o[DP / 8][4], m[2], l[2], cr[2];
    int stage = 0, first_tile = 0;
    bool fresh = true;  // the next tile begins a part
    for (long long u = u0; u < u1; ++u) {
        const int n = cur.len, row0 = cur.block * C::ROWS, rows = min(C::ROWS, n * G - row0), shift = cur.kv - n;
        if (fresh) {
            fresh = false;
            first_tile = cur.tile;
            // this warp's 16 rows of Q
            const float ks = head_scale(p.ks, cur.h);
            __syncwarp();
            for (int r = warp * 16; r < warp * 16 + 16; ++r) {
                const bool real = r < rows;
                const T *src = static_cast<const T *>(p.a.q) +
                               (real ? (long)(cur.start + (row0 + r) / G) * p.a.qs + (long)(cur.h * G + (row0 + r) % G) * D : 0);
                float x[DP / 32], amax = 0.f;
#pragma unroll
                for (int i = 0; i < DP / 32; ++i) {
                    const int d = lane + 32 * i;
                    x[i] = real && d < D ? to_f32(src[d]) : 0.f;
                    amax = fmaxf(amax, fabsf(x[i]));
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
                float back;
                const float power = kv4_row_power(amax, back) * p.sign;
#pragma unroll
                for (int i = 0; i < DP / 32; ++i) {
                    const int d = lane + 32 * i;
                    const uint32_t at = chunk_at<DP>(r, d / 8) + (d % 8) * 2;
                    const __half hi = __float2half_rn(x[i] * power);
                    *reinterpret_cast<__half *>(q_rows + at) = hi;
                    if constexpr (F32)
                        *reinterpret_cast<__half *>(q_rows + C::QBYTES + at) = __float2half_rn(x[i] * power - __half2float(hi));
                }
                if (lane == 0) s_c[r] = kv4_row_factor(p.c, back, ks);
            }
            __syncwarp();
            cr[0] = s_c[warp * 16 + g], cr[1] = s_c[warp * 16 + g + 8];
            m[0] = m[1] = -INFINITY, l[0] = l[1] = 0.f;
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        }
        copy_wait<STAGES - 2>();
        __syncthreads();  // the tile is here, and the last one's products are done
        {
            if (u_ahead < u1) {
                fetch(ahead, stage == 0 ? STAGES - 1 : stage - 1);
                if (++u_ahead < u1) advance(p, kList, ahead);
            }
            copy_commit();
        }
        // ---- codes to fp16, 16 channels at a time
        const unsigned char *from = smem + stage * 2 * C::RAW;
#pragma unroll 2
        for (int i = tid; i < 2 * KEYS * GR; i += C::THREADS) {
            const int which = i >= KEYS * GR, k = i - which * KEYS * GR, key = k / GR, grp = k % GR;
            const unsigned char *src = from + which * C::RAW;
            const uint2 w = *reinterpret_cast<const uint2 *>(src + k * 8);
            const uint32_t b = src[KEYS * GR * 8 + k], s = kv4_scales(b | b << 8);
            uint32_t d[2][4];
            kv4_codes(w.x, d[0]), kv4_codes(w.y, d[1]);
            unsigned char *to = tiles + which * C::TILE;
#pragma unroll
            for (int half = 0; half < 2; ++half)
                *reinterpret_cast<uint4 *>(to + chunk_at<DP>(key, grp * 2 + half)) =
                    make_uint4(mul_f16x2(d[half][0], s), mul_f16x2(d[half][1], s), mul_f16x2(d[half][2], s), mul_f16x2(d[half][3], s));
        }
        __syncthreads();
        // ---- scores of 16 rows
        const int j0 = cur.tile * KEYS;
        float s[KEYS / 8][4];
#pragma unroll
        for (int i = 0; i < KEYS / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) {
            uint32_t q[C::Q][4], k[4];
#pragma unroll
            for (int z = 0; z < C::Q; ++z)
                ldmatrix4(s_q + z * C::QBYTES + chunk_at<DP>(warp * 16 + (lane & 15), ks * 2 + (lane >> 4)), q[z]);
#pragma unroll
            for (int i = 0; i < KEYS / 16; ++i) {
                ldmatrix4(s_k + chunk_at<DP>(i * 16 + (lane >> 4) * 8 + (lane & 7), ks * 2 + ((lane >> 3) & 1)), k);
#pragma unroll
                for (int z = 0; z < C::Q; ++z) {
                    mma16816(s[2 * i], q[z], k[0], k[1]);
                    mma16816(s[2 * i + 1], q[z], k[2], k[3]);
                }
            }
        }
        // ---- running softmax of rows g and g + 8
        float mx[2] = {m[0], m[1]};
        const int rr = row0 + warp * 16 + g;
        const int seen[2] = {shift + rr / G + 1 - j0, shift + (rr + 8) / G + 1 - j0};
        const bool edge = j0 + KEYS > shift + row0 / G + 1;  // some row does not see the whole tile
        // (rows past the last hold zeros and see no more keys than there are)
        const int end = cur.kv - j0;
#pragma unroll
        for (int i = 0; i < KEYS / 8; ++i)
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                if (edge && i * 8 + t4 * 2 + (z & 1) >= min(seen[z >> 1], end)) s[i][z] = -INFINITY;
                mx[z >> 1] = fmaxf(mx[z >> 1], s[i][z]);
            }
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            mx[z] = fmaxf(mx[z], __shfl_xor_sync(0xffffffffu, mx[z], 1));
            mx[z] = fmaxf(mx[z], __shfl_xor_sync(0xffffffffu, mx[z], 2));
            if (mx[z] > m[z]) {
                // (a row that has seen nothing keeps l = o = 0 under any factor but NaN)
                const float f = m[z] == -INFINITY ? 1.f : exp2_fast((m[z] - mx[z]) * cr[z]);
                l[z] *= f;
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) o[i][2 * z] *= f, o[i][2 * z + 1] *= f;
                m[z] = mx[z];
            }
        }
        const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
        for (int i = 0; i < KEYS / 8; ++i)
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                s[i][z] = exp2_fast(fmaf(s[i][z] - base[z >> 1], cr[z >> 1], kShift));
                l[z >> 1] += s[i][z];
            }
        // ---- o += P V
#pragma unroll
        for (int i = 0; i < KEYS / 16; ++i) {
            uint32_t pa[C::Q][4];
            pa[0][0] = pack_f16(s[2 * i][0], s[2 * i][1]), pa[0][1] = pack_f16(s[2 * i][2], s[2 * i][3]);
            pa[0][2] = pack_f16(s[2 * i + 1][0], s[2 * i + 1][1]), pa[0][3] = pack_f16(s[2 * i + 1][2], s[2 * i + 1][3]);
            if constexpr (F32) {
                pa[1][0] = rest_f16(s[2 * i][0], s[2 * i][1], pa[0][0]), pa[1][1] = rest_f16(s[2 * i][2], s[2 * i][3], pa[0][1]);
                pa[1][2] = rest_f16(s[2 * i + 1][0], s[2 * i + 1][1], pa[0][2]);
                pa[1][3] = rest_f16(s[2 * i + 1][2], s[2 * i + 1][3], pa[0][3]);
            }
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) {
                uint32_t v[4];
                ldmatrix4_trans(s_v + chunk_at<DP>(i * 16 + (lane & 15), 2 * c + (lane >> 4)), v);
#pragma unroll
                for (int z = 0; z < C::Q; ++z) {
                    mma16816(o[2 * c], pa[z], v[0], v[1]);
                    mma16816(o[2 * c + 1], pa[z], v[2], v[3]);
                }
            }
        }
        stage = stage == STAGES - 1 ? 0 : stage + 1;

        const bool last = cur.tile + 1 == cur.tiles;
        if (last || u + 1 == u1) {
            // ---- the part ends
            fresh = true;
            const bool whole = last && first_tile == 0;
            if (last && tid == 0) {
                const long long first = u - cur.tile;  // the triple's first tile
                p.spans[span_of(p, cur)] = make_int2((int)(((first + 1) * ctas - 1) / U), (int)cta);
            }
            const float vs = head_scale(p.vs, cur.h);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                l[z] += __shfl_xor_sync(0xffffffffu, l[z], 1);
                l[z] += __shfl_xor_sync(0xffffffffu, l[z], 2);
                const int r = warp * 16 + g + 8 * z;
                if (r >= rows) continue;
                if (whole) {
                    const float inv = l[z] > 0.f ? 1.f / l[z] : l[z];  // (0 gives 0, NaN stays)
                    T *out = static_cast<T *>(p.a.out) + ((size_t)(cur.start + (row0 + r) / G) * p.a.H + cur.h * G + (row0 + r) % G) * D;
#pragma unroll
                    for (int i = 0; i < DP / 8; ++i)
                        if (i * 8 < D) store2(out + i * 8 + t4 * 2, o[i][2 * z] * inv * vs, o[i][2 * z + 1] * inv * vs);
                } else {
                    // a part that begins its triple is the CTA's last, any other its first
                    float *part = p.part + (2 * cta + (first_tile == 0)) * C::PART;
                    if (t4 == 0) part[r] = m[z], part[C::ROWS + r] = l[z], part[2 * C::ROWS + r] = cr[z];
                    part += 3 * C::ROWS + r * DP;
#pragma unroll
                    for (int i = 0; i < DP / 8; ++i)
                        *reinterpret_cast<float2 *>(part + i * 8 + t4 * 2) = make_float2(o[i][2 * z], o[i][2 * z + 1]);
                }
            }
        }
        advance(p, kList, cur);
    }
}

// ---------------------------------------------------------------- rows by the block of 8 or 16

// 16 x 5 drafts over 4096 keys, 16 heads of 256 on 2 (40 rows in three blocks): 37 us, against 80 for a tile of 64 rows.
//
// Rows are the columns of the products, keys and channels their rows: S^T = K Q^T and O^T = V^T P^T with 16 keys or 16
// channels to a tile, so that a cached value is converted into the registers of one product and no row
// of it is wasted on the few queries (8 to a column tile, NT of those).  Both contractions run over things that
// may be permuted: thread t of a quad takes the neighbouring channels [t DP/4, (t+1) DP/4) of its keys, group g of the warp the
// channels [g DP/8, (g+1) DP/8) of V, so that codes come from shared memory in wide loads; two keys' codes are
// interleaved by halves of bytes before they are converted, which pairs them as the second product needs.
//
// Every warp streams its own quarter of a tile's keys through two stages of its own and waits for no other
// warp before the end of a part.
template <int DP, int NT, typename T>
struct Narrow {
    static constexpr int WARP_KEYS = DP > 128 ? 32 : 64, KEYS = 4 * WARP_KEYS, ROWS = 8 * NT, THREADS = 128, STAGES = 2;
    static constexpr int KB = WARP_KEYS / 16;                // blocks of 16 keys
    static constexpr int Q = sizeof(T) == 4 ? 2 : 1;         // fp16 values to a query's
    static constexpr int RAW = WARP_KEYS * DP / 16 * 9;      // bytes of a warp's tile of K (or V): codes, then scales
    static constexpr bool QREG = Q * NT * DP <= 256;         // queries stay in registers, else in shared memory
    static constexpr int QBYTES = QREG ? 0 : Q * ROWS * DP * 2;
    static constexpr int SMEM = 4 * STAGES * 2 * RAW + 64 + QBYTES;  // (loads of channels past D may pass the end)
    static constexpr int PART = ROWS * (3 + DP);
    static constexpr int PER_SM = DP > 128 || NT * Q > 1 ? 2 : DP > 64 ? 3 : 4;
    static_assert(2 * RAW >= 8 * DP * 4, "a column tile's output fits a stage");
};

// The key of a block of 16 that is row m < 8 of the products' tiles (row m + 8: this one + 8).
__device__ __forceinline__ int key_of_row(int m) { return m & 1 ? 4 + ((m >> 1) ^ 1) : m >> 1; }

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// N words from shared memory that begin on a boundary of at least 8 bytes (WIDE: of their size).
template <int N, bool WIDE>
__device__ __forceinline__ void load_words(const unsigned char *at, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t *>(at);
    } else if constexpr (N == 2 || !WIDE) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint2 x = *reinterpret_cast<const uint2 *>(at + i * 4);
            w[i] = x.x, w[i + 1] = x.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(at + i * 4);
            w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
        }
    }
}
// N bytes, in one load if their place allows (WIDE).
template <int N, bool WIDE>
__device__ __forceinline__ uint32_t load_bytes(const unsigned char *at) {
    if constexpr (N == 1) return *at;
    else if constexpr (WIDE && N == 2) return *reinterpret_cast<const uint16_t *>(at);
    else if constexpr (WIDE) return *reinterpret_cast<const uint32_t *>(at);
    else {
        uint32_t x = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) x |= (uint32_t)at[i] << (8 * i);
        return x;
    }
}

template <int DP, int NT, typename T, bool FULL>
__global__ void __launch_bounds__(128, Narrow<DP, NT, T>::PER_SM) kv4_narrow_kernel(const Kv4Params p) {
    using C = Narrow<DP, NT, T>;
    constexpr int KEYS = C::KEYS, STAGES = C::STAGES, QN = C::Q, RAW = C::RAW;
    constexpr List kList = {C::ROWS, KEYS, 1};
    constexpr int KW = DP / 32, VW = DP / 64;  // words of a thread: of a key's channels, of a key's values
    constexpr int VS = DP > 128 ? 2 : 1;       // scales of a key's values
    constexpr int MT = DP / 16;                // tiles of channels, and steps of 16 channels
    constexpr bool F32 = sizeof(T) == 4;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float s_m[4][C::ROWS], s_l[4][C::ROWS], s_c[C::ROWS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    unsigned char *ring = smem + warp * STAGES * 2 * RAW;
    const uint32_t ring_at = sm100::smem_u32(ring);
    const int D = FULL ? DP : p.a.D, GR = D / 16, G = p.G;
    pdl_wait_primary();
    pdl_launch_dependents();  // (the joining blocks wait for this grid's end)
    long long u0, u1, U, ctas;
    Cursor cur;
    if (!find_run<C::THREADS>(p, kList, u0, u1, U, ctas, cur)) return;
    const long long cta = blockIdx.x;

    // The blocks of 16 keys of this warp's part of a tile: pages looked up a tile ahead.
    const int ps = p.a.page_size;
    const long page_bytes = (long)ps * GR * 9;
    const unsigned char *kc = static_cast<const unsigned char *>(p.a.k), *vc = static_cast<const unsigned char *>(p.a.v);
    auto split = [&](int key, int &index, int &at) {
        if (p.page_shift >= 0) index = key >> p.page_shift, at = key & (ps - 1);
        else index = key / ps, at = key - index * ps;
    };
    // (pages of several blocks of 16 keys are looked up by lane: lane i holds that of block i)
    auto look_up = [&](const Cursor &x) {
        const int key = x.tile * KEYS + warp * C::WARP_KEYS + min(lane, C::KB - 1) * 16;
        int index, at;
        split(key, index, at);
        return key < x.kv ? __ldg(p.a.block_table + (size_t)x.b * p.a.max_pages + index) : -1;
    };
    auto fetch = [&](const Cursor &x, int pages, int stage) {
        const uint32_t dst = ring_at + stage * 2 * RAW + lane * 16;
        const long between = vc - kc;
#pragma unroll
        for (int i = 0; i < C::KB; ++i) {
            const int page = __shfl_sync(0xffffffffu, pages, i);
            const bool read = page >= 0 && page < p.a.num_pages;
            int index, at;
            split(x.tile * KEYS + warp * C::WARP_KEYS + i * 16, index, at);
            // (nothing is read without a page; the addresses then lie in the cache's first block)
            const unsigned char *block = kc;
            if (read) block += ((long)page * p.a.HKV + x.h) * page_bytes;
            else at = 0;
            const unsigned char *codes = block + (at * GR * 8 + lane * 16);
#pragma unroll
            for (int c = 0; c < (FULL ? DP / 2 : 128); c += 32)
                if (FULL || c + lane < GR * 8) {
                    copy16(dst + (i * GR * 8 + c) * 16, codes + c * 16, read);
                    copy16(dst + RAW + (i * GR * 8 + c) * 16, codes + between + c * 16, read);
                }
            // lanes 0 to 15 bring K's scales, the others V's
            if ((lane & 15) < GR)
                copy16(dst + (lane < 16 ? 0 : RAW - 256) + (C::KB * GR * 8 + i * GR) * 16,
                       block + (lane < 16 ? 0 : between) + ((ps * 8 + at) * GR + (lane & 15) * 16), read);
        }
    };

    Cursor ahead = cur;
    int n_ahead = (int)min(u1 - u0, (long long)INT32_MAX), n_left = n_ahead;  // places to fetch, places to go
    auto to_tile = [&] {
        while (n_ahead > 0 && ahead.tile < 0) {
            advance(p, kList, ahead);
            --n_ahead;
        }
        return n_ahead > 0 ? look_up(ahead) : -1;
    };
    int pages = to_tile();
    auto fetch_next = [&](int stage) {
        if (n_ahead > 0) {
            fetch(ahead, pages, stage);
            --n_ahead;
            advance(p, kList, ahead);
            pages = to_tile();
        }
        copy_commit();
    };
#pragma unroll 1
    for (int i = 0; i < STAGES; ++i) fetch_next(i);

    // Queries as the second operand of the products: of step `ks`, two words of each lane.
    uint32_t q[C::QREG ? QN : 1][NT][C::QREG ? MT : 1][2];
    uint2 *s_q = reinterpret_cast<uint2 *>(smem + 4 * STAGES * 2 * RAW + 64);  // [QN][NT][MT][32]
    float o[NT][MT][4], m[NT][2], l[NT][2], cr[NT][2];
    int stage = 0, first_tile = 0;
    bool fresh = true;  // the next tile begins a part
#pragma unroll 1
    for (; n_left > 0; --n_left) {
        if (cur.tile < 0) {
            advance(p, kList, cur);
            continue;
        }
        const int n = cur.len, row0 = cur.block * C::ROWS, rows = min(C::ROWS, n * G - row0), shift = cur.kv - n;
        if (fresh) {
            fresh = false;
            first_tile = cur.tile;
            const float ks = head_scale(p.ks, cur.h);
            const auto load_rows = [&](int nt, auto put) {  // rows nt 8 + g, DP / 4 channels of each a thread
                const int r = nt * 8 + g;
                const T *src = static_cast<const T *>(p.a.q);
                if (r < rows) src += (long)(cur.start + (row0 + r) / G) * p.a.qs + (long)(cur.h * G + (row0 + r) % G) * D;
                float x[DP / 4], amax = 0.f;
                if (p.q_wide) {  // (D is a multiple of 16: no 16 bytes lie across its end)
                    constexpr int VEC = 16 / sizeof(T);
#pragma unroll
                    for (int i = 0; i < DP / 4; i += VEC) {
                        const int d = t4 * (DP / 4) + i;
                        Vec16<T> w;
                        w.u = make_uint4(0, 0, 0, 0);
                        if (r < rows && (FULL || d < D)) w.u = __ldg(reinterpret_cast<const uint4 *>(src + d));
#pragma unroll
                        for (int k = 0; k < VEC; ++k) x[i + k] = to_f32(w.v[k]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < DP / 4; ++i) {
                        const int d = t4 * (DP / 4) + i;
                        x[i] = r < rows && (FULL || d < D) ? to_f32(src[d]) : 0.f;
                    }
                }
#pragma unroll
                for (int i = 0; i < DP / 4; ++i) amax = fmaxf(amax, fabsf(x[i]));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                float back;
                const float power = kv4_row_power(amax, back) * p.sign;
#pragma unroll
                for (int i = 0; i < DP / 4; i += 4) {
                    const float y[4] = {x[i] * power, x[i + 1] * power, x[i + 2] * power, x[i + 3] * power};
                    const uint32_t hi[2] = {pack_f16(y[0], y[1]), pack_f16(y[2], y[3])};
                    put(0, i / 4, hi[0], hi[1]);
                    if constexpr (F32) put(1, i / 4, rest_f16(y[0], y[1], hi[0]), rest_f16(y[2], y[3], hi[1]));
                }
                return back;
            };
            if constexpr (C::QREG) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float back = load_rows(nt, [&](int z, int ks, uint32_t a, uint32_t b) { q[z][nt][ks][0] = a, q[z][nt][ks][1] = b; });
                    // this thread's columns are rows 2 t4 and 2 t4 + 1
                    const float factor = kv4_row_factor(p.c, back, ks);
                    cr[nt][0] = __shfl_sync(0xffffffffu, factor, t4 * 8), cr[nt][1] = __shfl_sync(0xffffffffu, factor, t4 * 8 + 4);
                }
            } else {
                if (warp < NT) {
                    const float back = load_rows(warp, [&](int z, int ks, uint32_t a, uint32_t b) { s_q[((z * NT + warp) * MT + ks) * 32 + lane] = make_uint2(a, b); });
                    if (t4 == 0) s_c[warp * 8 + g] = kv4_row_factor(p.c, back, ks);
                }
                __syncthreads();
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) cr[nt][0] = s_c[nt * 8 + t4 * 2], cr[nt][1] = s_c[nt * 8 + t4 * 2 + 1];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
                for (int i = 0; i < MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
            }
        }
        copy_wait<STAGES - 1>();
        __syncwarp();  // the warp's keys are here

        const int j0 = cur.tile * KEYS + warp * C::WARP_KEYS;
        const unsigned char *kt = ring + stage * 2 * RAW, *vt = kt + RAW;
        if (j0 < cur.kv) {
            // ---- scores
            float s[NT][C::KB][4];
#pragma unroll
            for (int kb = 0; kb < C::KB; ++kb) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[nt][kb][0] = s[nt][kb][1] = s[nt][kb][2] = s[nt][kb][3] = 0.f;
                uint32_t w[2][KW], sc[2][DP / 64];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int key = kb * 16 + y * 8 + key_of_row(g);
                    load_words<KW, FULL>(kt + key * (D / 2) + t4 * (DP / 8), w[y]);
                    const uint32_t b = load_bytes<DP / 64, FULL>(kt + C::WARP_KEYS * (D / 2) + key * GR + t4 * (DP / 64));
#pragma unroll
                    for (int i = 0; i < DP / 64; i += 2) {
                        const uint32_t two = kv4_scales(i ? b >> 16 : b);
                        sc[y][i] = __byte_perm(two, 0, 0x1010);
                        if (i + 1 < DP / 64) sc[y][i + 1] = __byte_perm(two, 0, 0x3232);
                    }
                }
#pragma unroll
                for (int i = 0; i < KW; ++i) {  // eight channels, two steps
                    uint32_t lo[4], hi[4];
                    kv4_codes(w[0][i], lo), kv4_codes(w[1][i], hi);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t a[4] = {mul_f16x2(lo[2 * y], sc[0][i / 2]), mul_f16x2(hi[2 * y], sc[1][i / 2]),
                                               mul_f16x2(lo[2 * y + 1], sc[0][i / 2]), mul_f16x2(hi[2 * y + 1], sc[1][i / 2])};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int z = 0; z < QN; ++z) {
                                if constexpr (C::QREG) {
                                    mma16816(s[nt][kb], a, q[z][nt][2 * i + y][0], q[z][nt][2 * i + y][1]);
                                } else {
                                    const uint2 b = s_q[((z * NT + nt) * MT + 2 * i + y) * 32 + lane];
                                    mma16816(s[nt][kb], a, b.x, b.y);
                                }
                            }
                    }
                }
            }
            // ---- running softmax: this thread's rows 2 t4 and 2 t4 + 1, its keys of key_of_row(g)
            const bool edge = j0 + C::WARP_KEYS > shift + row0 / G + 1;  // some row does not see all of these
            uint32_t pt[QN][NT][C::KB][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (edge)
#pragma unroll
                    for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const int key = j0 + kb * 16 + (z >> 1) * 8 + key_of_row(g), r = row0 + nt * 8 + t4 * 2 + (z & 1);
                            if (key >= min(cur.kv, shift + r / G + 1)) s[nt][kb][z] = -INFINITY;
                        }
                float f[2], base[2];
                bool moved = false;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float mx = fmaxf(s[nt][0][y], s[nt][0][y + 2]);
#pragma unroll
                    for (int kb = 1; kb < C::KB; ++kb) mx = fmaxf(mx, fmaxf(s[nt][kb][y], s[nt][kb][y + 2]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(fmaxf(mx, m[nt][y]), __shfl_xor_sync(0xffffffffu, mx, 16));
                    // (a row that has seen nothing keeps l = o = 0 under any factor but NaN)
                    f[y] = m[nt][y] == -INFINITY ? 1.f : exp2_fast((m[nt][y] - mx) * cr[nt][y]);
                    moved |= mx > m[nt][y];
                    m[nt][y] = mx;
                    base[y] = mx == -INFINITY ? 0.f : mx;
                }
                if (__any_sync(0xffffffffu, moved)) {
                    l[nt][0] *= f[0], l[nt][1] *= f[1];
#pragma unroll
                    for (int i = 0; i < MT; ++i) o[nt][i][0] *= f[0], o[nt][i][1] *= f[1], o[nt][i][2] *= f[0], o[nt][i][3] *= f[1];
                }
#pragma unroll
                for (int kb = 0; kb < C::KB; ++kb) {
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        s[nt][kb][z] = exp2_fast(fmaf(s[nt][kb][z] - base[z & 1], cr[nt][z & 1], kShift));
                        l[nt][z & 1] += s[nt][kb][z];
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float a = s[nt][kb][2 * y], b = s[nt][kb][2 * y + 1];
                        const uint32_t hi = pack_f16(a, b);
                        pt[0][nt][kb][y] = transposed(hi);
                        if constexpr (F32) pt[1][nt][kb][y] = transposed(rest_f16(a, b, hi));
                    }
                }
            }
            // ---- O^T += V^T P^T
#pragma unroll
            for (int kb = 0; kb < C::KB; ++kb) {
                uint32_t w[4][VW], sc[2][VS];
                const unsigned char *vs = vt + C::WARP_KEYS * (D / 2);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint32_t b[2];
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const int key = kb * 16 + y * 8 + (z ? 4 + (t4 ^ 1) : t4);  // rows 2 t4 and 2 t4 + 1
                        load_words<VW, FULL>(vt + key * (D / 2) + g * (DP / 16), w[2 * y + z]);
                        b[z] = load_bytes<VS, FULL>(vs + key * GR + g * (DP / 8) / 16);
                    }
                    sc[y][0] = kv4_scales(__byte_perm(b[0], b[1], 0x0040));
                    if constexpr (DP > 128) sc[y][1] = kv4_scales(__byte_perm(b[0], b[1], 0x0051));
                }
#pragma unroll
                for (int i = 0; i < VW; ++i) {
                    uint32_t even[2][4], odd[2][4];  // of two neighbouring keys, the channels of a word
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t a = w[2 * y][i], b = w[2 * y + 1][i];
                        kv4_codes((a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u), even[y]);
                        kv4_codes(((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u), odd[y]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t s0 = sc[0][i / 2], s1 = sc[1][i / 2];
                        const uint32_t a[4] = {mul_f16x2(even[0][j], s0), mul_f16x2(odd[0][j], s0), mul_f16x2(even[1][j], s1),
                                               mul_f16x2(odd[1][j], s1)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int z = 0; z < QN; ++z) mma16816(o[nt][4 * i + j], a, pt[z][nt][kb][0], pt[z][nt][kb][1]);
                    }
                }
            }
        }

        const bool last = cur.tile + 1 == cur.tiles;
        if (last || n_left == 1) {
            // ---- the part ends: the warps' outputs meet in their stages, which are free now
            fresh = true;
            const bool whole = last && first_tile == 0;
            if (last && tid == 0) {
                const long long first = u1 - n_left - cur.tile;  // the place of the triple's first tile
                p.spans[span_of(p, cur)] = make_int2((int)(((first + 1) * ctas - 1) / U), (int)cta);
            }
            const float vs = head_scale(p.vs, cur.h);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[nt][y] += __shfl_xor_sync(0xffffffffu, l[nt][y], d);
                    if (g == 0) s_m[warp][nt * 8 + t4 * 2 + y] = m[nt][y], s_l[warp][nt * 8 + t4 * 2 + y] = l[nt][y];
                }
            __syncthreads();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float f[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int r = nt * 8 + t4 * 2 + y;
                    const float M = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
                    float L = 0.f;
#pragma unroll
                    for (int w = 0; w < 4; ++w) L += s_m[w][r] == -INFINITY ? s_l[w][r] : s_l[w][r] * exp2_fast((s_m[w][r] - M) * cr[nt][y]);
                    f[y] = m[nt][y] == -INFINITY ? 1.f : exp2_fast((m[nt][y] - M) * cr[nt][y]);
                    m[nt][y] = M, l[nt][y] = L;
                }
                float *mine = reinterpret_cast<float *>(ring + stage * 2 * RAW);  // [8][DP]
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        *reinterpret_cast<float2 *>(mine + (t4 * 2 + y) * DP + g * (DP / 8) + 2 * i) =
                            make_float2(o[nt][i][y] * f[y], o[nt][i][y + 2] * f[y]);
                __syncthreads();
                // a warp to two rows
                const float *all = reinterpret_cast<const float *>(smem + stage * 2 * RAW);
                constexpr int NEXT = STAGES * 2 * RAW / 4;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int row = warp * 2 + y, r = nt * 8 + row;
                    if (r >= rows) continue;
                    float M, L, c;  // from a thread that has this row's column
                    {
                        const int from = warp;  // (t4 of column 2 warp + y)
                        M = __shfl_sync(0xffffffffu, m[nt][y], from), L = __shfl_sync(0xffffffffu, l[nt][y], from);
                        c = __shfl_sync(0xffffffffu, cr[nt][y], from);
                    }
                    const float inv = L > 0.f ? 1.f / L : L;  // (0 gives 0, NaN stays)
                    float *part = p.part + (2 * cta + (first_tile == 0)) * C::PART;
                    T *out = static_cast<T *>(p.a.out) + ((size_t)(cur.start + (row0 + r) / G) * p.a.H + cur.h * G + (row0 + r) % G) * D;
                    if (!whole && lane == 0) part[r] = M, part[C::ROWS + r] = L, part[2 * C::ROWS + r] = c;
#pragma unroll
                    for (int d = lane * 2; d < DP; d += 64) {
                        float2 x = make_float2(0.f, 0.f);
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const float2 v = *reinterpret_cast<const float2 *>(all + w * NEXT + row * DP + d);
                            x.x += v.x, x.y += v.y;
                        }
                        if (!whole) *reinterpret_cast<float2 *>(part + 3 * C::ROWS + r * DP + d) = x;
                        else if (FULL || d < D) store2(out + d, x.x * inv * vs, x.y * inv * vs);
                    }
                }
                __syncthreads();  // read, before the next column tile's or the copies to come
            }
        }
        __syncwarp();  // the warp is done with this stage
        fetch_next(stage);
        stage = stage == STAGES - 1 ? 0 : stage + 1;
        advance(p, kList, cur);
    }
}

// ---------------------------------------------------------------- parts

// Joins the parts of each triple that several CTAs shared.  With many triples, of few parts each, a warp to a row; with few, of
// many, eight warps, which go by every eighth part and meet in shared memory.  A running maximum lets the parts be loaded
// before any other is known.  (What the first kernel did not write is read before its end.)
template <int DP, typename T, int WARPS>
__global__ void __launch_bounds__(WARPS == 1 ? 128 : WARPS * 32) kv4_join_kernel(const Kv4Params p, int rows) {
    constexpr int E = DP / 32, N = 4;  // channels of a lane, parts loaded at a time
    constexpr int AT_ONCE = WARPS == 1 ? 4 : 1;  // rows of a block
    __shared__ float s_m[WARPS], s_l[WARPS], s_o[WARPS == 1 ? 1 : WARPS][DP];
    const int tid = threadIdx.x, lane = tid & 31, warp = WARPS == 1 ? 0 : tid >> 5;
    const int h = blockIdx.x % p.a.HKV, block = blockIdx.x / p.a.HKV % p.blocks, b = blockIdx.x / p.a.HKV / p.blocks;
    int start, len, kv;
    if (block >= seq_blocks(p, rows, b, start, len, kv)) {
        // (a grid none of whose blocks waits could end before the first kernel, and let the next call begin beside that)
        if (blockIdx.x == 0 && blockIdx.y == 0) pdl_wait_primary();
        return;
    }
    const float vs = head_scale(p.vs, h);
    pdl_wait_primary();
    const int2 span = p.spans[blockIdx.x];
    if (span.x == span.y) return;
    const int PART = rows * (3 + DP);
    auto part = [&](int c) { return p.part + (2L * c + (c == span.x)) * PART; };
    for (int r0 = blockIdx.y * AT_ONCE; r0 < rows; r0 += gridDim.y * AT_ONCE) {
        const int r = WARPS == 1 ? r0 + (tid >> 5) : r0;
        const long row = (long)block * rows + r;
        if (r >= rows || row >= (long)len * p.G) return;
        const float c_row = part(span.x)[2 * rows + r];
        float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = 0.f;
        for (int c0 = span.x + warp; c0 <= span.y; c0 += N * WARPS) {
            float pm[N], pl[N];
            float2 po[N][E / 2];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const bool real = c0 + k * WARPS <= span.y;
                const float *x = part(real ? c0 + k * WARPS : c0);
                pm[k] = real ? x[r] : -INFINITY, pl[k] = x[rows + r];
                x += 3 * rows + r * DP + lane * E;
#pragma unroll
                for (int i = 0; i < E / 2; ++i) po[k][i] = reinterpret_cast<const float2 *>(x)[i];
            }
            float M = m;
#pragma unroll
            for (int k = 0; k < N; ++k) M = fmaxf(M, pm[k]);
            const float f = m == -INFINITY ? 0.f : exp2_fast((m - M) * c_row);
            l *= f;
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] *= f;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                // (a part that saw no key has l = o = 0; NaN, of a row whose query is not finite, has m = -inf too)
                const bool real = c0 + k * WARPS <= span.y;
                const float w = pm[k] == -INFINITY ? (real && pl[k] != 0.f ? 1.f : 0.f) : exp2_fast((pm[k] - M) * c_row);
                l = fmaf(w, pl[k], l);
#pragma unroll
                for (int i = 0; i < E / 2; ++i)
                    o[2 * i] = fmaf(w, po[k][i].x, o[2 * i]), o[2 * i + 1] = fmaf(w, po[k][i].y, o[2 * i + 1]);
            }
            m = M;
        }
        T *out = static_cast<T *>(p.a.out) + ((size_t)(start + row / p.G) * p.a.H + h * p.G + row % p.G) * p.a.D;
        if constexpr (WARPS == 1) {
            const float inv = l > 0.f ? 1.f / l : l;  // (0 gives 0, NaN stays)
            if (lane * E < p.a.D)
#pragma unroll
                for (int i = 0; i < E; i += 2) store2(out + lane * E + i, o[i] * inv * vs, o[i + 1] * inv * vs);
        } else {
            if (lane == 0) s_m[warp] = m;
            __syncthreads();
            float M = s_m[0];
#pragma unroll
            for (int w = 1; w < WARPS; ++w) M = fmaxf(M, s_m[w]);
            const float f = m == -INFINITY ? (l != 0.f ? 1.f : 0.f) : exp2_fast((m - M) * c_row);
#pragma unroll
            for (int i = 0; i < E; ++i) s_o[warp][lane * E + i] = o[i] * f;
            if (lane == 0) s_l[warp] = l * f;
            __syncthreads();
            float L = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) L += s_l[w];
            const float inv = L > 0.f ? 1.f / L : L;  // (0 gives 0, NaN stays)
            for (int d = tid; d < p.a.D; d += WARPS * 32) {
                float x = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) x += s_o[w][d];
                out[d] = from_f32<T>(x * inv * vs);
            }
            __syncthreads();  // the sums have been read
        }
    }
}

// ---------------------------------------------------------------- host

int padded(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
// (the most that any of the kernels asks for: blocks of 8 rows)
size_t span_bytes(int B, int HKV, long blocks) { return ((size_t)B * blocks * HKV * 8 + 255) & ~size_t(255); }
// Rows of the parts of one SM's CTAs, at most.
constexpr int part_rows(int DP) { return 64 * 256 / DP; }
long row_blocks(int H, int HKV, int max_q, int rows) { return ((long)max_q * (H / HKV) + rows - 1) / rows; }

// Sequences of up to so many rows run in blocks of 8 or 16, which convert the cache anew; the tcgen05 kernel takes more
// rows at once, but needs items for its SMs.  With a pair of (sequence, head) to every half SM it has them (64 requests over
// U[1, 4096], 8 key-value heads: 32 rows of heads of 128 take 120 us in blocks and 118 there, 40 174 and 120; 20 rows of heads of 256
// 222 and 189).  With fewer pairs the blocks' even runs win up to three blocks (2 requests over U[1, 65536]: 48 rows of
// heads of 128 71 us and 74, 64 rows 89 and 75; of heads of 64 65 and 62; 8 requests over U[1, 8192]: 42 and 50, 52 and 57,
// 38 and 48).
constexpr int kNarrowRows = kSplitRows;
int narrow_rows(const Attn &a, int dtype) {
    if (dtype != GDN_BF16) return kNarrowRows;
    if ((long)a.B * a.HKV >= 2 * 152) return a.D > 128 ? 16 : 32;
    return a.D > 64 ? 48 : kNarrowRows;
}

// A kernel over the sequences of its rows (C: its sizes), then the join of what several CTAs shared.
template <int DP, typename T, typename C>
cudaError_t launch_kernels(void (*kernel)(Kv4Params), Kv4Params p, void *ws, cudaStream_t s) {
    static_assert(C::PER_SM * C::ROWS <= part_rows(DP), "parts of an SM's CTAs");
    p.blocks = (int)((std::min((long)p.a.max_q * p.G, (long)p.max_rows) + C::ROWS - 1) / C::ROWS);
    p.spans = static_cast<int2 *>(ws);
    p.part = reinterpret_cast<float *>(static_cast<char *>(ws) + span_bytes(p.a.B, p.a.HKV, p.blocks));
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const long triples = (long)p.a.B * p.blocks * p.a.HKV;
    if (triples > INT32_MAX) return cudaErrorInvalidConfiguration;
    const long most = triples * (((long)p.a.max_pages * p.a.page_size + C::KEYS - 1) / C::KEYS);
    const long grid = std::min((long)C::PER_SM * std::min(sms, kMaxSms), most);
    cudaError_t e = launch_kernel(kernel, dim3((unsigned)grid), dim3(C::THREADS), C::SMEM, s, true, p);
    note_launch();
    if (e != cudaSuccess) return e;
    // Few triples have many parts each, many have few: then a warp to a row, and with many blocks several rows to each (most
    // of them have nothing to join, and leaving takes its time too).
    const long rows = std::min((long)p.a.max_q * p.G, (long)C::ROWS), few = triples * 2 <= sms;
    const dim3 blocks((unsigned)triples, (unsigned)std::min(few ? rows : (rows + 3) / 4, std::max(1L, 4096 / triples)));
    e = few ? launch_kernel(kv4_join_kernel<DP, T, 8>, blocks, dim3(256), 0, s, true, p, C::ROWS)
            : launch_kernel(kv4_join_kernel<DP, T, 1>, blocks, dim3(128), 0, s, true, p, C::ROWS);
    note_launch();
    return e;
}

template <int DP, typename T>
cudaError_t launch_wide(Kv4Params p, int min_rows, void *ws, cudaStream_t s) {
    using C = Wide<DP, T>;
    static std::atomic<uint64_t> attr_set{0};
    const cudaError_t e = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(kv4_wide_kernel<DP, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e != cudaSuccess) return e;
    p.min_rows = min_rows, p.max_rows = INT32_MAX;
    return launch_kernels<DP, T, C>(kv4_wide_kernel<DP, T>, p, ws, s);
}

template <int DP, int NT, typename T, bool FULL>
cudaError_t launch_narrow(Kv4Params p, void *ws, cudaStream_t s) {
    using C = Narrow<DP, NT, T>;
    static std::atomic<uint64_t> attr_set{0};
    const cudaError_t e = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(kv4_narrow_kernel<DP, NT, T, FULL>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e != cudaSuccess) return e;
    p.min_rows = 0, p.max_rows = narrow_rows(p.a, sizeof(T) == 2 ? GDN_BF16 : GDN_F32);
    return launch_kernels<DP, T, C>(kv4_narrow_kernel<DP, NT, T, FULL>, p, ws, s);
}

template <int DP, typename T>
cudaError_t launch_rows(const Kv4Params &p, void *ws, cudaStream_t s) {
    const long rows = (long)p.a.max_q * p.G;
    const bool full = p.a.D == DP;
    cudaError_t e = cudaSuccess;
    const int most = narrow_rows(p.a, sizeof(T) == 2 ? GDN_BF16 : GDN_F32);
    if (p.G <= most) {
        // (a batch of single tokens beside longer slices: blocks of 8 if those hold them; wide fp32 heads: 16 rows would not
        // fit the registers)
        const bool one = rows <= 8 || (rows > most && p.G <= 8) || (DP > 128 && sizeof(T) == 4);
        if (one) {
            e = full ? launch_narrow<DP, 1, T, true>(p, ws, s) : launch_narrow<DP, 1, T, false>(p, ws, s);
        } else if constexpr (DP <= 128 || sizeof(T) == 2) {
            e = full ? launch_narrow<DP, 2, T, true>(p, ws, s) : launch_narrow<DP, 2, T, false>(p, ws, s);
        }
    }
    if (e != cudaSuccess || rows <= most) return e;
    if constexpr (sizeof(T) == 4) {
        return launch_wide<DP, T>(p, most, ws, s);
    } else {
        Attn a = p.a;
        a.part = static_cast<float *>(ws), a.out_scale = p.vs;
        return launch_attention_prompt_kv4(a, p.ks, most, s);
    }
}

template <typename T>
cudaError_t launch(const Kv4Params &p, void *ws, cudaStream_t s) {
    switch (padded(p.a.D)) {
    case 64: return launch_rows<64, T>(p, ws, s);
    case 128: return launch_rows<128, T>(p, ws, s);
    default: return launch_rows<256, T>(p, ws, s);
    }
}

}  // namespace

size_t attention_kv4_workspace(int B, int N, int H, int HKV, int D, int max_q) {
    const long blocks = std::max(row_blocks(H, HKV, max_q, 64), row_blocks(H, HKV, std::min(max_q, kNarrowRows), 8));
    const size_t parts = span_bytes(B, HKV, blocks) + 2 * (size_t)kMaxSms * part_rows(padded(D)) * (3 + padded(D)) * 4;
    Attn a{};
    a.B = B, a.HKV = HKV, a.D = D;
    const bool slices = (long)max_q * (H / HKV) > narrow_rows(a, GDN_BF16);
    return std::max(parts, slices ? attention_prompt_part_floats(B, N, H, HKV, D, max_q) * 4 : 0);
}

cudaError_t launch_attention_kv4(const Attn &a, const float *k_scale, const float *v_scale, int dtype, void *ws, cudaStream_t s) {
    Kv4Params p{};
    p.a = a;
    p.ks = k_scale, p.vs = v_scale;
    p.G = a.H / a.HKV;
    p.c = std::fabs(a.scale) * kLog2e;
    p.sign = a.scale < 0.f ? -1.f : 1.f;
    p.q_wide = rows_aligned(a.q, a.qs, a.D, dtype == GDN_BF16 ? 2 : 4);
    p.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (a.page_size == 1 << i) p.page_shift = i;
    return dtype == GDN_BF16 ? launch<__nv_bfloat16>(p, ws, s) : launch<float>(p, ws, s);
}

}  // namespace gdn
