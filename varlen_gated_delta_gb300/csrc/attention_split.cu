// attention_split.cu - attention of few new tokens over long paged histories
// (decode steps, drafted tokens): bf16, at most 64 (token, head of a group) rows
// to a sequence and key-value head.
//
// Every key and value is read once for all rows that share it, and each takes
// only 4 operations a row and channel: bound by HBM at 4 D bytes a key and
// key-value head.  So the work is cut by bytes, not by rows: the 64-key tiles of
// all (sequence, key-value head) pairs form one list, and every CTA takes an
// equal run of it.  A run may begin and end inside a pair; such a CTA leaves the
// running maximum m, the sum l and an unscaled output of its part, and a second
// kernel joins the parts of a pair: with M = max m_i, o = sum o_i 2^(m_i - M) /
// sum l_i 2^(m_i - M).  Which parts exist follows from the lengths alone, so the
// result does not depend on timing.
//
// Key and value rows stream through a ring of tiles filled by 16-byte cp.async
// copies (their slots are looked up once a key, by lane).  The products are 16-row
// mma.sync: with rows this few they are far from binding, and registers hold
// scores, probabilities and output without the staging that larger tiles need.
// With up to 16 rows the four warps share out the keys of a tile, with more they
// form row groups; warps that share rows join at the end of a part through shared
// memory.
//
// 16 requests of 16384 tokens, 32 heads of 128 on 8, one token each: 161 us, 6.7
// TB/s, the measured copy's rate.  Short steps are bound by the launches and the
// dependent loads before the first tile (one request of 64 tokens: 7.5 us), and
// the most rows of wide heads by latency: their registers leave eight warps to an SM,
// which wait for fragments, products and copies in turn (16 x 5 drafts over 4096 keys,
// 16 heads of 256 on 2, 40 rows in 64: 62 us, 2.2 TB/s, tensor pipe 29% active).  Leaving
// out the row group without rows, sharing twelve units of three groups evenly among
// the schedulers, and looking key slots up a tile ahead gave 62, 65 and 64 us.
#include <cmath>

#include "attention.cuh"
#include "sm100.cuh"

namespace gdn {
namespace {

constexpr int kKeys = 64;
constexpr int kMaxCtas = 3 * 160;

struct SplitParams {
    Attn a;
    int G;
    float c;      // |scale| log2(e)
    int negate;   // scale < 0
    int2 *spans;  // [B * HKV]: first and last CTA of a pair
    float *part;  // [2 * CTAs][ROWS * (2 + DP)]
};

template <int DP, int MT>
struct Split {
    static constexpr int ROWS = 16 * MT;       // padded rows of a pair
    // Wide heads leave one CTA to an SM: with rows for it, eight warps instead of four hide each
    // other's latency (16 x 5 drafts over 4096 keys, 16 heads of 256 on 2: 65 -> 62 us).
    static constexpr int WARPS = DP > 128 && MT > 1 ? 8 : 4, THREADS = WARPS * 32;
    static constexpr int WK = WARPS / MT;      // warps that share the keys of a tile
    static constexpr int COPY = kKeys / WARPS; // keys that a warp copies of a tile
    static constexpr int KW = kKeys / WK;      // keys of a warp in a tile
    static constexpr int STAGES = 3;
    static constexpr int HALF = kKeys * DP * 2;  // bytes of a K (or V) tile
    // Q rows (bf16); at the end of a part, half of the channels of the joined output (fp32)
    static constexpr int Q_BYTES = ROWS * DP * 2;
    static constexpr bool QREG = DP <= 128;      // Q fragments stay in registers
    // With one row group Q comes with its part's first tile, in the same stage, so that a part
    // begins without a load of its own to wait for (64 x U[1, 8192] keys, 32 heads of 128 on 8: 166 -> 160 us).
    static constexpr bool QSTAGE = QREG && MT == 1;
    static constexpr int SMEM = STAGES * 2 * HALF + (QSTAGE ? 1 + STAGES : 1) * Q_BYTES;
    static constexpr int PER_SM = DP > 128 ? 1 : DP > 64 ? 2 : 3;  // CTAs that fit
    static constexpr int PART = ROWS * (2 + DP);  // floats of a part: m, l, o
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
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
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
// Byte offset of 16-byte chunk c of row r: chunks of 8 neighbouring rows fall into different banks.
template <int DP>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return (uint32_t)(r * DP * 2 + ((c ^ (r & 7)) << 4));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Key tiles of one key-value head of sequence b; 0: not ours.
__device__ __forceinline__ int pair_tiles(const SplitParams &p, int rows, int b, int &start, int &len, int &kv) {
    if (b >= p.a.B || !attn_seq(p.a, b, start, len, kv) || len == 0 || (long)len * p.G > rows) return 0;
    return kv > 0 ? (kv + kKeys - 1) / kKeys : 1;  // (no keys: one tile that gives zeros)
}

// A place in the list of tiles.
struct Cursor {
    int b, h, tile, tiles, start, len, kv;
};

template <int DP, int MT>
__global__ void __launch_bounds__(Split<DP, MT>::THREADS) attn_split_kernel(const SplitParams p) {
    using C = Split<DP, MT>;
    constexpr int CH = DP / 8, WK = C::WK, KW = C::KW, STAGES = C::STAGES, kThreads = C::THREADS;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long s_scan[C::WARPS];
    __shared__ long long s_first;
    __shared__ Cursor s_cur;
    __shared__ int s_bad[3];  // of this part, the last and the next
    __shared__ float s_ml[C::WARPS][2][16];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const int mt = warp / WK, wk = warp % WK;  // this warp's rows and keys
    const uint32_t ring = sm100::smem_u32(smem), s_q = ring + STAGES * 2 * C::HALF;
    float *s_sum = reinterpret_cast<float *>(smem + STAGES * 2 * C::HALF);  // [ROWS][DP / 2]
    const int D = p.a.D, G = p.G, HKV = p.a.HKV;
    pdl_wait_primary();
    pdl_launch_dependents();  // (the joining blocks wait for this grid's end)

    // ---- this CTA's run of tiles [u0, u1): threads own neighbouring sequences
    const int per = (p.a.B + kThreads - 1) / kThreads;
    long long mine = 0;
    Cursor own;  // (with one sequence a thread, all that is read of it)
    for (int i = 0; i < per; ++i) {
        own.b = tid * per + i;
        mine += own.tiles = pair_tiles(p, C::ROWS, own.b, own.start, own.len, own.kv);
    }
    long long sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += x;
    }
    if (lane == 31) s_scan[warp] = sum;
    if (tid < 3) s_bad[tid] = 0;
    __syncthreads();
    long long all = 0;
    for (int w = 0; w < C::WARPS; ++w) {
        if (w < warp) sum += s_scan[w];
        all += s_scan[w];
    }
    // every CTA that takes part has at least one tile
    const long long U = all * HKV, ctas = U < gridDim.x ? U : gridDim.x, cta = blockIdx.x;
    if (cta >= ctas) return;
    const long long u0 = cta * U / ctas, u1 = (cta + 1) * U / ctas;
    {
        long long at = (sum - mine) * HKV;
        if (u0 >= at && u0 < sum * HKV)
            for (int i = 0; i < per; ++i) {
                if (per > 1) {
                    own.b = tid * per + i;
                    own.tiles = pair_tiles(p, C::ROWS, own.b, own.start, own.len, own.kv);
                }
                const long long n = (long long)own.tiles * HKV;
                if (u0 < at + n) {
                    s_cur = own, s_first = at;
                    break;
                }
                at += n;
            }
    }
    __syncthreads();
    Cursor cur = s_cur;
    cur.h = (int)((u0 - s_first) / cur.tiles);
    cur.tile = (int)((u0 - s_first) % cur.tiles);
    auto advance = [&](Cursor &x) {
        if (++x.tile < x.tiles) return;
        x.tile = 0;
        if (++x.h < HKV) return;
        x.h = 0;
        do x.tiles = pair_tiles(p, C::ROWS, ++x.b, x.start, x.len, x.kv);
        while (x.tiles == 0 && x.b < p.a.B);
    };

    // ---- copies: warp w brings keys COPY w .. COPY (w + 1) - 1 of a tile
    const __nv_bfloat16 *kc = static_cast<const __nv_bfloat16 *>(p.a.k), *vc = static_cast<const __nv_bfloat16 *>(p.a.v);
    auto load_q = [&](const Cursor &x, uint32_t dst) {  // asynchronous; without the sign of a negative scale
        for (int i = tid; i < C::ROWS * CH; i += kThreads) {
            const int r = i / CH, c = i % CH;
            const bool read = r < x.len * G && c * 8 < D;
            const long e = read ? (long)(x.start + r / G) * p.a.qs + (long)(x.h * G + r % G) * D + c * 8 : 0;
            copy16(dst + chunk_at<DP>(r, c), static_cast<const __nv_bfloat16 *>(p.a.q) + e, read);
        }
    };
    auto fetch = [&](const Cursor &x, int stage, bool first) {
        if (C::QSTAGE && (first || x.tile == 0)) load_q(x, s_q + (1 + stage) * C::Q_BYTES);
        const int key = x.tile * kKeys + warp * C::COPY + (lane & (C::COPY - 1));
        long row = -1;
        if (key < x.kv) row = attn_key_row(p.a, x.b, x.start, key, p.a.ks);
        const uint32_t kd = ring + stage * 2 * C::HALF, vd = kd + C::HALF;
        constexpr int RPI = 32 / CH > 0 ? 32 / CH : 1;  // rows a warp copies at a time
#pragma unroll
        for (int i = 0; i < C::COPY / RPI; ++i) {
            const int r = i * RPI + (CH < 32 ? lane / CH : 0), c = lane % CH;
            const long at = __shfl_sync(0xffffffffu, row, r);
            const bool read = at >= 0 && c * 8 < D;
            const long e = read ? at + (long)x.h * D + c * 8 : 0;
            copy16(kd + chunk_at<DP>(warp * C::COPY + r, c), kc + e, read);
            copy16(vd + chunk_at<DP>(warp * C::COPY + r, c), vc + e, read);
        }
    };

    Cursor ahead = cur;
    long long u_ahead = u0;
    for (int i = 0; i < STAGES - 1; ++i) {
        if (u_ahead < u1) {
            fetch(ahead, i, i == 0);
            ++u_ahead;
            if (u_ahead < u1) advance(ahead);
        }
        copy_commit();
    }

    uint32_t qf[C::QREG ? DP / 16 : 1][4];
    float o[DP / 8][4], m[2], l[2];
    int stage = 0;
    bool fresh = true;   // the next tile begins a part
    int first_tile = 0;  // of this part
    int bad_at = 0;      // its place in s_bad
    for (long long u = u0; u < u1; ++u) {
        const int n = cur.len, rows = n * G, shift = cur.kv - n;
        const bool begins = fresh;
        if (begins) {
            fresh = false;
            first_tile = cur.tile;
            if constexpr (!C::QSTAGE) {
                __syncthreads();  // the last part's use of this place is over
                for (int i = tid; i < C::ROWS * CH; i += kThreads) {
                    const int r = i / CH, c = i % CH;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (r < rows && c * 8 < D) {
                        x = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.a.q) +
                                                                  (long)(cur.start + r / G) * p.a.qs + (long)(cur.h * G + r % G) * D + c * 8));
                        if (p.negate) x.x ^= 0x80008000u, x.y ^= 0x80008000u, x.z ^= 0x80008000u, x.w ^= 0x80008000u;
                    }
                    *reinterpret_cast<uint4 *>(smem + STAGES * 2 * C::HALF + chunk_at<DP>(r, c)) = x;
                }
                __syncthreads();
            }
            bad_at = bad_at == 2 ? 0 : bad_at + 1;
            if (tid == 0) s_bad[bad_at == 2 ? 0 : bad_at + 1] = 0;  // (two parts ago: read by all)
            m[0] = m[1] = -INFINITY, l[0] = l[1] = 0.f;
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        }
        copy_wait<STAGES - 2>();
        __syncthreads();  // the tile is here, and the slot that is filled next is free
        if (C::QREG && begins) {
            const uint32_t q = s_q + (C::QSTAGE ? (1 + stage) * C::Q_BYTES : 0);
#pragma unroll
            for (int ks = 0; ks < (C::QREG ? DP / 16 : 0); ++ks) {
                ldmatrix4(q + chunk_at<DP>(mt * 16 + (lane & 15), ks * 2 + (lane >> 4)), qf[ks]);
                if (C::QSTAGE && p.negate)
#pragma unroll
                    for (int z = 0; z < 4; ++z) qf[ks][z] ^= 0x80008000u;
            }
        }
        {
            const int next = stage == 0 ? STAGES - 1 : stage - 1;
            if (u_ahead < u1) {
                fetch(ahead, next, false);
                ++u_ahead;
                if (u_ahead < u1) advance(ahead);
            }
            copy_commit();
        }
        const uint32_t kd = ring + stage * 2 * C::HALF, vd = kd + C::HALF;
        const int j0 = cur.tile * kKeys;
        const bool edge = j0 + kKeys > shift + 1;  // some row does not see the whole tile
        if (edge && n > 1) {
            // values that some row must not see: non-finite ones become 0 and join their rows at the end
            const int r0 = max(0, shift + 1 - j0), r1 = min(kKeys, cur.kv - j0);
            for (int i = tid; i < max(0, r1 - r0) * CH; i += kThreads) {
                uint32_t *w = reinterpret_cast<uint32_t *>(smem + stage * 2 * C::HALF + C::HALF + chunk_at<DP>(r0 + i / CH, i % CH));
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const uint32_t x = w[z];
                    const bool lo = (x & 0x7f80u) == 0x7f80u, hi = (x & 0x7f800000u) == 0x7f800000u;
                    if (lo | hi) w[z] = x & (lo ? 0xffff0000u : 0xffffffffu) & (hi ? 0x0000ffffu : 0xffffffffu), s_bad[bad_at] = 1;
                }
            }
            __syncthreads();
        }
        // ---- scores of 16 rows and KW keys
        float s[KW / 8][4];
#pragma unroll
        for (int i = 0; i < KW / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
        // (fragments are loaded one step ahead of the products that use them, here and below)
        uint32_t qa[2][4], kb[2][KW / 16][4];
        auto load_qk = [&](int ks) {
            if constexpr (!C::QREG)
                ldmatrix4(s_q + chunk_at<DP>(mt * 16 + (lane & 15), ks * 2 + (lane >> 4)), qa[ks & 1]);
#pragma unroll
            for (int i = 0; i < KW / 16; ++i)
                ldmatrix4(kd + chunk_at<DP>(wk * KW + i * 16 + (lane >> 4) * 8 + (lane & 7), ks * 2 + ((lane >> 3) & 1)),
                          kb[ks & 1][i]);
        };
        load_qk(0);
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) {
            if (ks + 1 < DP / 16) load_qk(ks + 1);
#pragma unroll
            for (int i = 0; i < KW / 16; ++i) {
                const uint32_t(&q)[4] = C::QREG ? qf[C::QREG ? ks : 0] : qa[ks & 1];
                mma16816(s[2 * i], q, kb[ks & 1][i][0], kb[ks & 1][i][1]);
                mma16816(s[2 * i + 1], q, kb[ks & 1][i][2], kb[ks & 1][i][3]);
            }
        }
        // ---- running softmax of rows g and g + 8
        float mx[2] = {m[0], m[1]};
        const int rr = mt * 16 + g;
        const int seen[2] = {shift + rr / G + 1 - j0, shift + (rr + 8) / G + 1 - j0};
#pragma unroll
        for (int i = 0; i < KW / 8; ++i)
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                if (edge && wk * KW + i * 8 + t4 * 2 + (z & 1) >= seen[z >> 1]) s[i][z] = -INFINITY;
                mx[z >> 1] = fmaxf(mx[z >> 1], s[i][z]);
            }
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            mx[z] = fmaxf(mx[z], __shfl_xor_sync(0xffffffffu, mx[z], 1));
            mx[z] = fmaxf(mx[z], __shfl_xor_sync(0xffffffffu, mx[z], 2));
        }
        if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
            // (a row that has seen nothing keeps l = o = 0 under any factor but NaN)
            const float f0 = m[0] == -INFINITY ? 1.f : exp2_fast((m[0] - mx[0]) * p.c);
            const float f1 = m[1] == -INFINITY ? 1.f : exp2_fast((m[1] - mx[1]) * p.c);
            l[0] *= f0, l[1] *= f1;
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) o[i][0] *= f0, o[i][1] *= f0, o[i][2] *= f1, o[i][3] *= f1;
            m[0] = mx[0], m[1] = mx[1];
        }
        const float b0 = m[0] == -INFINITY ? 0.f : -m[0] * p.c, b1 = m[1] == -INFINITY ? 0.f : -m[1] * p.c;
#pragma unroll
        for (int i = 0; i < KW / 8; ++i) {
            s[i][0] = exp2_fast(fmaf(s[i][0], p.c, b0)), s[i][1] = exp2_fast(fmaf(s[i][1], p.c, b0));
            s[i][2] = exp2_fast(fmaf(s[i][2], p.c, b1)), s[i][3] = exp2_fast(fmaf(s[i][3], p.c, b1));
            l[0] += s[i][0] + s[i][1];
            l[1] += s[i][2] + s[i][3];
        }
        // ---- o += P V: a step is 16 keys and four blocks of eight channels
        constexpr int STEPS = KW / 16 * (CH / 4);
        uint32_t vb[2][2][4];
        auto load_v = [&](int step) {
            const int i = step / (CH / 4), c = step % (CH / 4) * 4;
#pragma unroll
            for (int y = 0; y < 2; ++y)
                ldmatrix4_trans(vd + chunk_at<DP>(wk * KW + i * 16 + (lane & 15), c + 2 * y + (lane >> 4)), vb[step & 1][y]);
        };
        load_v(0);
#pragma unroll
        for (int step = 0; step < STEPS; ++step) {
            const int i = step / (CH / 4), c = step % (CH / 4) * 4;
            if (step + 1 < STEPS) load_v(step + 1);
            const uint32_t pa[4] = {pack_bf16(s[2 * i][0], s[2 * i][1]), pack_bf16(s[2 * i][2], s[2 * i][3]),
                                    pack_bf16(s[2 * i + 1][0], s[2 * i + 1][1]), pack_bf16(s[2 * i + 1][2], s[2 * i + 1][3])};
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                mma16816(o[c + 2 * y], pa, vb[step & 1][y][0], vb[step & 1][y][1]);
                mma16816(o[c + 2 * y + 1], pa, vb[step & 1][y][2], vb[step & 1][y][3]);
            }
        }
        stage = stage == STAGES - 1 ? 0 : stage + 1;

        const bool last = cur.tile + 1 == cur.tiles;
        if (last || u + 1 == u1) {
            // ---- the part ends: join the warps that share rows, then write the pair or the part
            fresh = true;
            const bool whole = last && first_tile == 0;
            if (last && tid == 0) {
                const long long pair = u - cur.tile;  // the pair's first tile
                p.spans[cur.b * HKV + cur.h] = make_int2((int)(((pair + 1) * ctas - 1) / U), (int)cta);
            }
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                l[z] += __shfl_xor_sync(0xffffffffu, l[z], 1);
                l[z] += __shfl_xor_sync(0xffffffffu, l[z], 2);
            }
            if (WK > 1) {
                if (t4 == 0) {
#pragma unroll
                    for (int z = 0; z < 2; ++z) s_ml[warp][0][g + 8 * z] = m[z], s_ml[warp][1][g + 8 * z] = l[z];
                }
                __syncthreads();
                float f[2];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    float M = -INFINITY, L = 0.f;
#pragma unroll
                    for (int w = 0; w < WK; ++w) M = fmaxf(M, s_ml[mt * WK + w][0][g + 8 * z]);
#pragma unroll
                    for (int w = 0; w < WK; ++w) {
                        const float mw = s_ml[mt * WK + w][0][g + 8 * z], lw = s_ml[mt * WK + w][1][g + 8 * z];
                        L += mw == -INFINITY ? lw : lw * exp2_fast((mw - M) * p.c);
                    }
                    f[z] = m[z] == -INFINITY ? 1.f : exp2_fast((m[z] - M) * p.c);
                    m[z] = M, l[z] = L;
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int w = 0; w < WK; ++w) {
                        if (wk == w) {
#pragma unroll
                            for (int i = 0; i < DP / 16; ++i)
#pragma unroll
                                for (int z = 0; z < 2; ++z) {
                                    float(&v)[4] = o[half * (DP / 16) + i];
                                    float2 *at = reinterpret_cast<float2 *>(s_sum + (mt * 16 + g + 8 * z) * (DP / 2) + i * 8 + t4 * 2);
                                    float2 x = make_float2(v[2 * z] * f[z], v[2 * z + 1] * f[z]);
                                    if (w > 0) x.x += at->x, x.y += at->y;
                                    if (w == WK - 1) v[2 * z] = x.x, v[2 * z + 1] = x.y;
                                    else *at = x;
                                }
                        }
                        __syncthreads();
                    }
                }
            }
            if (wk == WK - 1) {  // this warp holds the joined rows mt 16 + g, + 8
                const bool bad = s_bad[bad_at] != 0;
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int r = mt * 16 + g + 8 * z;
                    if (r >= rows) continue;
                    if (bad) {
                        const int end = min(cur.kv, shift + r / G + 1);
                        for (int j = max(first_tile * kKeys, shift + 1); j < min(end, j0 + kKeys); ++j) {
                            const long at = attn_key_row(p.a, cur.b, cur.start, j, p.a.vs);
                            if (at < 0) continue;
#pragma unroll
                            for (int i = 0; i < DP / 8; ++i)
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const int d = i * 8 + t4 * 2 + y;
                                    const float v = d < D ? __bfloat162float(vc[at + (long)cur.h * D + d]) : 0.f;
                                    if (!isfinite(v)) o[i][2 * z + y] += v;
                                }
                        }
                    }
                    if (whole) {
                        const float inv = l[z] > 0.f ? 1.f / l[z] : (l[z] == 0.f ? 0.f : l[z]);  // (NaN stays)
                        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.a.out) +
                                             ((size_t)(cur.start + r / G) * p.a.H + cur.h * G + r % G) * D;
#pragma unroll
                        for (int i = 0; i < DP / 8; ++i)
                            if (i * 8 < D)
                                *reinterpret_cast<uint32_t *>(out + i * 8 + t4 * 2) =
                                    pack_bf16(o[i][2 * z] * inv, o[i][2 * z + 1] * inv);
                    } else {
                        // a part that begins its pair is the CTA's last, any other its first
                        float *part = p.part + (2 * cta + (first_tile == 0)) * C::PART;
                        if (t4 == 0) part[r] = m[z], part[C::ROWS + r] = l[z];
                        part += 2 * C::ROWS + r * DP;
#pragma unroll
                        for (int i = 0; i < DP / 8; ++i)
                            *reinterpret_cast<float2 *>(part + i * 8 + t4 * 2) = make_float2(o[i][2 * z], o[i][2 * z + 1]);
                    }
                }
            }
        }
        advance(cur);
    }
}

// Joins the parts of each pair that several CTAs shared: a block to a (pair, row).
template <int DP, int MT>
__global__ void __launch_bounds__(128) attn_split_join_kernel(const SplitParams p) {
    using C = Split<DP, MT>;
    const int b = blockIdx.x / p.a.HKV, h = blockIdx.x % p.a.HKV, r = blockIdx.y;
    pdl_wait_primary();
    int start, len, kv;
    const int2 span = p.spans[blockIdx.x];  // (written for the pairs of valid sequences only)
    if (pair_tiles(p, C::ROWS, b, start, len, kv) == 0 || r >= len * p.G || span.x == span.y) return;
    auto part = [&](int c) { return p.part + (2L * c + (c == span.x)) * C::PART; };
    // every part's weight first (a history over many CTAs has many parts), then the weighted sum
    __shared__ float s_w[kMaxCtas], s_red[2][4];
    const int tid = threadIdx.x, n = span.y - span.x + 1;
    float M = -INFINITY, L = 0.f;
    for (int i = tid; i < n; i += 128) M = fmaxf(M, part(span.x + i)[r]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    if ((tid & 31) == 0) s_red[0][tid >> 5] = M;
    __syncthreads();
    M = fmaxf(fmaxf(s_red[0][0], s_red[0][1]), fmaxf(s_red[0][2], s_red[0][3]));
    for (int i = tid; i < n; i += 128) {
        const float *x = part(span.x + i);
        const float mc = x[r], f = mc == -INFINITY ? 1.f : exp2_fast((mc - M) * p.c);
        s_w[i] = f;
        L += x[C::ROWS + r] * f;
    }
    L = group_sum<32>(L);
    if ((tid & 31) == 0) s_red[1][tid >> 5] = L;
    __syncthreads();
    L = s_red[1][0] + s_red[1][1] + s_red[1][2] + s_red[1][3];
    const float inv = L > 0.f ? 1.f / L : L;  // (0 gives 0, NaN stays)
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.a.out) +
                         ((size_t)(start + r / p.G) * p.a.H + h * p.G + r % p.G) * p.a.D;
    for (int d = tid; d < p.a.D; d += 128) {
        float o = 0.f;
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
            const float f = s_w[i], v = part(span.x + i)[2 * C::ROWS + r * DP + d];
            o += f > 0.f ? v * f : 0.f;  // (a part that counts for nothing may hold inf)
        }
        out[d] = __float2bfloat16_rn(L != 0.f ? o * inv : 0.f);
    }
}

size_t span_bytes(int B, int HKV) { return ((size_t)B * HKV * 8 + 255) & ~size_t(255); }

template <int DP, int MT>
cudaError_t launch(const Attn &a, void *ws, cudaStream_t s) {
    using C = Split<DP, MT>;
    static std::atomic<uint64_t> attr_set{0};
    cudaError_t e = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(attn_split_kernel<DP, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e != cudaSuccess) return e;
    SplitParams p{};
    p.a = a;
    p.G = a.H / a.HKV;
    p.c = std::fmax(std::fabs(a.scale) * kLog2e, 1e-30f);
    p.negate = a.scale < 0.f;
    p.spans = static_cast<int2 *>(ws);
    p.part = reinterpret_cast<float *>(static_cast<char *>(ws) + span_bytes(a.B, a.HKV));
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const long slots = (long)sms * C::PER_SM;
    const long most = (long)a.B * a.HKV * (((long)a.max_pages * a.page_size + kKeys - 1) / kKeys);
    long grid = slots < kMaxCtas ? slots : kMaxCtas;
    if (most < grid) grid = most;
    if ((long)a.B * a.HKV > INT32_MAX) return cudaErrorInvalidConfiguration;
    e = launch_kernel(attn_split_kernel<DP, MT>, dim3((unsigned)grid), dim3(C::THREADS), C::SMEM, s, true, p);
    note_launch();
    if (e != cudaSuccess) return e;
    const long rows = (long)a.max_q * p.G < C::ROWS ? (long)a.max_q * p.G : C::ROWS;
    e = launch_kernel(attn_split_join_kernel<DP, MT>, dim3((unsigned)(a.B * a.HKV), (unsigned)rows), dim3(128), 0, s,
                      true, p);
    note_launch();
    return e;
}

template <int DP>
cudaError_t launch_rows(const Attn &a, void *ws, cudaStream_t s) {
    const long rows = (long)a.max_q * (a.H / a.HKV);
    if (rows <= 16) return launch<DP, 1>(a, ws, s);
    if (rows <= 32) return launch<DP, 2>(a, ws, s);
    return launch<DP, 4>(a, ws, s);
}

}  // namespace

bool attention_split_supported(const Attn &a, int dtype) {
    return dtype == GDN_BF16 && a.block_table != nullptr && a.H / a.HKV <= kSplitRows && rows_aligned(a.q, a.qs, a.D, 2) &&
           rows_aligned(a.k, a.ks, a.D, 2) && rows_aligned(a.v, a.vs, a.D, 2) && ((uintptr_t)a.out & 15) == 0;
}

size_t attention_split_workspace(int B, int H, int HKV, int D, int max_q) {
    const long rows = (long)max_q * (H / HKV);
    const int R = rows <= 16 ? 16 : rows <= 32 ? 32 : 64, dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
    return span_bytes(B, HKV) + 2 * (size_t)kMaxCtas * R * (2 + dp) * 4;
}

cudaError_t launch_attention_split(const Attn &a, void *ws, cudaStream_t s) {
    if (a.D <= 64) return launch_rows<64>(a, ws, s);
    if (a.D <= 128) return launch_rows<128>(a, ws, s);
    return launch_rows<256>(a, ws, s);
}

}  // namespace gdn
