// The shared prefix's part of the decode attention on the tensor cores (tcgen05, TMA),
// sm_100a.
//
// For one KV head the queries of the whole batch are one tall matrix (n_seq n_tok G
// rows), so the prefix is read once for up to 256 of them and the two products run as
// M = 128 tensor-core tiles.  A CTA takes (KV head, key split, 256 rows): two streams
// of 128 rows share the K/V tiles of the split; with 128 rows or fewer both streams
// hold the same rows and take the even and the odd key tiles, joined at the end.
// Consecutive CTAs hold the row tiles of one key split, so the re-reads of its keys
// meet in L2.
//
// Warps: 0-7 and 8-15 are the streams' softmax (two threads per row, half of a tile's
// keys each), 16 loads K/V tiles by TMA into a ring, 17 issues the products.  Per stream
// and key tile: S = Q K^T to tensor memory; the softmax threads read their rows, keep a
// running maximum m that is raised only when a row outgrows it by 2^8 (O is rescaled in
// tensor memory then, a rare event), and write P = 2^(S - m) over the S columns; O += P V
// takes P from tensor memory.  While one stream's softmax runs, the other's products do.
// m starts as the exact fp32 maximum of the row's first tile, so that a weight of 1 or
// more always exists however large the logits are: a bound rounded to bf16 exceeds logits
// of 2^14 by more than the exponent's 126 and loses every weight of the row.
//
// Bound: up to 256 rows per KV head by memory (134 MB of K/V for 64 sequences with 4 heads
// to a group: 41 us, of which 27 are the tiles at 5.5 TB/s), beyond that by the tensor
// cores: the main loop runs at 1.27 PFLOP/s (256 sequences, 8 heads to a group, 4 KV heads,
// 16384 keys: 54 us and about 13 us of start and end).  One thread per row instead of two
// ran as fast but held a whole row of S; issuing the products from lane 0 under an
// ordinary branch cost a fifth (100 us against 79 at the time); O of a tile and S of the
// next go out together, because the tensor core idles while the issuing thread waits.
//
// P is bf16: one rounding for a bf16 output; three bf16 parts (24 bits) for an f32
// output, over key tiles of 64 so that the parts fit beside S.
#include "cache.cuh"
#include "tc.cuh"

namespace crs {

constexpr int kPfThreads = 576;
constexpr int kPfRows = 256;                     // rows of a CTA: two streams of 128
constexpr uint64_t kPfWaitNs = 1000000000ull;    // 1 s: a wait that long means a fault
constexpr int kPfSpare = 3 * 1024;               // bytes for the tiles' alignment, PfTop and PfBars
constexpr float kPfSlack = 8.0f;                 // log2 units a logit may exceed the running shift

template <int D, bool SPLIT> struct PfCfg {
    static constexpr int kKeys = SPLIT ? 64 : 128;           // keys per tile
    static constexpr int kParts = SPLIT ? 3 : 1;             // bf16 parts of P
    static constexpr int kTile = kKeys * D * 2;              // bytes of a K or V tile
    static constexpr int kQ = 128 * D * 2;                   // bytes of a Q tile
    static constexpr int kStages = kTile >= 32768 ? 5 : 8;   // >= 5: see the order of use below
    static constexpr int kTiles = 2 * kQ + kStages * kTile;
    static constexpr int kSmem = kTiles + kPfSpare;
    // tensor memory columns: S and the P over it, the parts of P that S cannot hold, O
    static constexpr int kPCols = kKeys / 2;
    static __host__ __device__ constexpr int s_col(int u) { return u * (SPLIT ? 128 : kKeys); }
    static __host__ __device__ constexpr int o_col(int u) { return 256 + u * D; }
};
static_assert(PfCfg<128, false>::kStages * PfCfg<128, false>::kTile >= 2 * 128 * 128 * 4 &&
                  PfCfg<128, true>::kStages * PfCfg<128, true>::kTile >= 2 * 128 * 128 * 4 &&
                  PfCfg<64, true>::kStages * PfCfg<64, true>::kTile >= 2 * 128 * 64 * 4,
              "the results are staged in the ring");

struct PfBars {
    uint64_t q_full, kv_full[8], kv_empty[8], s_full[2], p_full[2][2], o_full[2], drain;
    uint32_t tmem;
    int abort;
};
typedef float PfTop[2][2][128];                  // [stream][half of a tile's keys][row]: maxima
// All of it is dynamic shared memory: the tiles start `lead` bytes in, on a 1024-byte
// boundary, PfTop follows them, PfBars take the lead where they fit there, else the end.
// With a static part the tiles of D = 128 and bf16 output would not fit beside PfTop.
static_assert(1008 + sizeof(PfTop) <= kPfSpare && sizeof(PfBars) + sizeof(PfTop) + sizeof(PfBars) <= kPfSpare,
              "PfTop always fits behind the tiles, PfBars before them or behind PfTop");

// 2^x of two values on the FMA pipe, for a part of the weights, because the exponential
// unit alone (16 a clock and SM) takes as long as the products: Cody and Waite's reduction
// x = n + f, |f| <= 1/2 (n by adding and subtracting 1.5 2^23), a minimax polynomial of
// degree 4 for 2^f (largest relative error 2.7e-6 as evaluated, fitted by reweighted least
// squares on Chebyshev nodes), and n added to the exponent.  x below kPfPolyLeast becomes
// it: there n = -127, the polynomial of f = 2^-17 is 33 steps above 1, and its exponent
// field ends at 0, so the value is 33 2^-149, which is 0 in bf16: a key too far to count
// adds nothing, however large its V.  Between it and 2^-126 the value is off by up to 2^-127.
constexpr int kPfPoly = 2;                       // of 8 pairs
constexpr float kPfPolyLeast = -127.0f + 0x1p-17f;
__device__ __forceinline__ float2 pf_exp2_poly(float2 x) {
    x.x = fmax_nan(x.x, kPfPolyLeast);
    x.y = fmax_nan(x.y, kPfPolyLeast);
    const float2 magic = make_float2(12582912.0f, 12582912.0f);
    const float2 t = __fadd2_rn(x, magic);
    const float2 n = __fadd2_rn(t, make_float2(-12582912.0f, -12582912.0f));
    const float2 f = __ffma2_rn(n, make_float2(-1.0f, -1.0f), x);
    float2 p = make_float2(0x1.3997d6p-7f, 0x1.3997d6p-7f);
    p = __ffma2_rn(p, f, make_float2(0x1.ca1440p-5f, 0x1.ca1440p-5f));
    p = __ffma2_rn(p, f, make_float2(0x1.ec06dap-3f, 0x1.ec06dap-3f));
    p = __ffma2_rn(p, f, make_float2(0x1.62e0dcp-1f, 0x1.62e0dcp-1f));
    p = __ffma2_rn(p, f, make_float2(0x1.ffffe8p-1f, 0x1.ffffe8p-1f));
    p.x = __uint_as_float(__float_as_uint(p.x) + (__float_as_uint(t.x) << 23));
    p.y = __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(t.y) << 23));
    return p;
}

static_assert(PfCfg<128, false>::kSmem <= 232448 && PfCfg<128, true>::kSmem <= 232448 &&
                  PfCfg<64, false>::kSmem <= 232448 && PfCfg<64, true>::kSmem <= 232448,
              "shared memory of one CTA");

__device__ __forceinline__ float pf_max3(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// the query of row R of KV head h's tall matrix (null past the last row), and whether its
// token exists (known later than the address)
__device__ __forceinline__ const __nv_bfloat16 *pf_query(const CaArgs &a, int h, int R, bool &exists) {
    exists = false;
    if (R >= a.c.n_seq * a.M) return nullptr;
    const int s = R / a.M, r = R - s * a.M, i = r / a.G, g = r - i * a.G;
    exists = i < cache_new(a.c, a.n_new, a.n_tok, s, cache_len(a.c, s));
    return a.Q + (((size_t)s * a.n_tok + i) * a.n_q + h * a.G + g) * a.c.D;
}

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kPfThreads, 1)
cache_prefix_kernel(CaArgs a, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    using C = PfCfg<D, SPLIT>;
    constexpr int KT = C::kKeys;
    extern __shared__ __align__(16) unsigned char pf_raw[];
    const uint32_t lead = (1024u - (smem_u32(pf_raw) & 1023u)) & 1023u;
    unsigned char *sQ = pf_raw + lead;
    unsigned char *ring = sQ + 2 * C::kQ;
    PfTop &row_top = *reinterpret_cast<PfTop *>(sQ + C::kTiles);
    PfBars &B = *reinterpret_cast<PfBars *>(lead >= sizeof(PfBars) ? pf_raw : sQ + C::kTiles + sizeof(PfTop));
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);      // uniform for the compiler too
    dependents_may_start();

    const int mt = blockIdx.x % a.tc_tiles, rest = blockIdx.x / a.tc_tiles;
    const int split = rest % a.tc_splits, h = rest / a.tc_splits;
    const int rows = a.c.n_seq * a.M;
    const int row0 = mt * kPfRows;
    const bool pair = rows - row0 <= 128;        // both streams hold the same rows
    const int PT = (a.prefix_len + KT - 1) / KT;
    const int t0 = (int)((long long)split * PT / a.tc_splits), t1 = (int)((long long)(split + 1) * PT / a.tc_splits);
    const int n = t1 - t0;                       // key tiles of this split (>= 1)
    auto count_of = [&](int u) { return pair ? (n + 1 - u) / 2 : n; };
    auto tile_of = [&](int u, int i) { return pair ? 2 * i + u : i; };

    if (tid == 0) {
        tc::mbar_init(&B.q_full, 512);
        for (int i = 0; i < C::kStages; ++i) {
            tc::mbar_init(&B.kv_full[i], 1);
            tc::mbar_init(&B.kv_empty[i], 1);
        }
        for (int u = 0; u < 2; ++u) {
            tc::mbar_init(&B.s_full[u], 1);
            tc::mbar_init(&B.p_full[u][0], 4);
            tc::mbar_init(&B.p_full[u][1], 4);
            tc::mbar_init(&B.o_full[u], 1);
        }
        tc::mbar_init(&B.drain, 1);
        B.abort = 0;
        tc::mbar_fence_init();
    }
    if (warp == 0) tc::tmem_alloc(&B.tmem, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = B.tmem;
    volatile int *abort_flag = &B.abort;
    auto wait = [&](uint64_t *bar, uint32_t parity, uint32_t site, bool forceable) {
        const bool ok = tc::mbar_wait_bounded(bar, parity & 1u, kPfWaitNs, K_CACHE_PREFIX, site, 10000u, forceable,
                                              abort_flag);
        if (!ok) *abort_flag = 1;
        return ok;
    };

    if (warp == 16) {
        // ---- K_0, V_0, K_1, V_1, ... through the ring
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(&tm_k) : "memory");
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(&tm_v) : "memory");
            int issued = 0;
            for (; issued < 2 * n; ++issued) {
                const int st = issued % C::kStages, use = issued / C::kStages;
                if (use > 0 && !wait(&B.kv_empty[st], (uint32_t)(use - 1), 2, false)) break;
                tc::mbar_arrive_expect_tx(&B.kv_full[st], C::kTile);
                const void *map = (issued & 1) ? (const void *)&tm_v : (const void *)&tm_k;
                unsigned char *dst = ring + st * C::kTile;
                const int key = (t0 + (issued >> 1)) * KT;
#pragma unroll
                for (int hh = 0; hh < D / 64; ++hh)
                    tc::tma_load_3d(dst + hh * KT * 128, map, hh * 64, h, key, &B.kv_full[st]);
            }
            // no copy may still be on its way when the CTA leaves, after an early end too
            for (int k = max(0, issued - C::kStages); k < issued; ++k)
                tc::mbar_wait_bounded(&B.kv_full[k % C::kStages], (uint32_t)(k / C::kStages) & 1u, kPfWaitNs,
                                      K_CACHE_PREFIX, 3);
        }
        __syncwarp();
    } else if (warp == 17) {
        // ---- products.  Order of use of the ring: K_0 (K_1), then per step V_i, K_{i+1}
        // of each stream; a tile is released when the last product that reads it completes.
        constexpr uint32_t id_s = tc::idesc_bf16_f32(128, KT, 0, 0), id_o = tc::idesc_bf16_f32(128, D, 0, 1);
        const uint64_t q_desc = tc::smem_desc(smem_u32(sQ), 16, 1024, tc::kLayoutSW128);
        const uint64_t k_desc = tc::smem_desc(smem_u32(ring), 16, 1024, tc::kLayoutSW128);
        const uint64_t v_desc = tc::smem_desc(smem_u32(ring), KT * 128, 1024, tc::kLayoutSW128);
        if (tc::elect_one()) {
            // S of stream u's tile i; releases K unless the other stream still needs it
            auto issue_s = [&](int u, int i) {
                const int st = 2 * tile_of(u, i) % C::kStages;
                const uint64_t qd = q_desc + (uint64_t)(pair ? 0 : u * (C::kQ >> 4));
                const uint64_t kd = k_desc + (uint64_t)(st * (C::kTile >> 4));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc::mma_bf16(tmem + C::s_col(u), qd + (kk >> 2) * (128 * 128 >> 4) + (kk & 3) * 2,
                                 kd + (kk >> 2) * (KT * 128 >> 4) + (kk & 3) * 2, id_s, kk > 0 ? 1u : 0u);
                tc::commit(&B.s_full[u]);
                if (pair || u == 1) tc::commit(&B.kv_empty[st]);
            };
            auto wait_kv = [&](int k, uint32_t site) {
                return wait(&B.kv_full[k % C::kStages], (uint32_t)(k / C::kStages), site, false);
            };
            bool ok = wait(&B.q_full, 0, 5, false);
            for (int u = 0; ok && u < 2; ++u) {
                if (count_of(u) == 0) continue;
                ok = wait_kv(2 * tile_of(u, 0), 4);
                tc::fence_after();
                if (ok) issue_s(u, 0);
            }
            // O of tile i, then S of tile i + 1, in one go: waiting between them would leave the
            // tensor core idle.  Streams on the same rows take tiles in turn, and their next K
            // tile may still be on its way: there O goes first.
            const int steps = count_of(0);       // the longer stream
            for (int i = 0; ok && i < steps; ++i) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (!ok || i >= count_of(u)) continue;
                    const int k = 2 * tile_of(u, i) + 1, st = k % C::kStages;
                    const bool more = i + 1 < count_of(u);
                    if (pair || u == 0) ok = wait_kv(k, 6) && (pair || !more || wait_kv(k + 1, 4));
                    const uint64_t vd = v_desc + (uint64_t)(st * (C::kTile >> 4));
                    auto issue_o = [&](int k0, int k1) {
                        tc::fence_after();
#pragma unroll
                        for (int part = 0; part < C::kParts; ++part)
#pragma unroll
                            for (int kk = k0; kk < k1; ++kk)
                                tc::mma_f16_ts(tmem + C::o_col(u),
                                               tmem + (uint32_t)(C::s_col(u) + part * C::kPCols + kk * 8),
                                               vd + kk * (16 * 128 >> 4), id_o,
                                               (i > 0 || kk > 0 || part > 0) ? 1u : 0u);
                    };
                    ok = ok && wait(&B.p_full[u][0], (uint32_t)i, 7, false);
                    if (ok) issue_o(0, KT / 32);
                    ok = ok && wait(&B.p_full[u][1], (uint32_t)i, 7, false);
                    if (!ok) continue;
                    issue_o(KT / 32, KT / 16);
                    if (!more) tc::commit(&B.o_full[u]);
                    if (!pair && more) issue_s(u, i + 1);
                    if (pair || u == 1) tc::commit(&B.kv_empty[st]);
                    if (pair && more) {
                        ok = wait_kv(2 * tile_of(u, i + 1), 4);
                        tc::fence_after();
                        if (ok) issue_s(u, i + 1);
                    }
                }
            }
            if (!ok) {                           // let what was issued finish
                tc::commit(&B.drain);
                tc::mbar_wait_bounded(&B.drain, 0, kPfWaitNs, K_CACHE_PREFIX, 8);
            }
        }
        __syncwarp();
    } else {
        // ---- softmax: stream u, half hh of a tile's keys, row r of the stream's 128
        constexpr int HK = KT / 2, HD = D / 2;
        const int u = warp >> 3, hh = (warp >> 2) & 1, quad = warp & 3, r = quad * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const int row = row0 + (pair ? r : u * 128 + r);
        // the two warps of a row meet once per tile on a barrier of their own; one that gives up
        // arrives there, so that the other is not left waiting (and gives up at the next tile,
        // whose S cannot come without both halves of P)
        const int meet_id = 1 + u * 4 + quad;
        auto meet = [&]() { asm volatile("bar.sync %0, 64;\n" ::"r"(meet_id) : "memory"); };
        {
            // the stream's query rows, one half of D per thread (streams on the same rows: a quarter);
            // a negative scale goes into their signs, which is exact
            const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
            unsigned char *dst = sQ + (pair ? 0 : u * C::kQ);
            bool exists;
            const uint4 *q = reinterpret_cast<const uint4 *>(pf_query(a, h, row, exists));
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                if (pair && part != u) continue;
                uint4 w[D / 32];
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    w[c] = q ? q[(hh * 2 + part) * (D / 32) + c] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    if (!exists) w[c] = make_uint4(0u, 0u, 0u, 0u);
                    w[c].x ^= flip; w[c].y ^= flip; w[c].z ^= flip; w[c].w ^= flip;
                    const int at = (hh * 2 + part) * (D / 32) + c;
                    *reinterpret_cast<uint4 *>(dst + (at >> 3) * 128 * 128 + tc::sw128(r, at & 7)) = w[c];
                }
            }
            tc::fence_proxy_async();
            tc::mbar_arrive(&B.q_full);
        }
        // never 0, so that a masked -inf stays one (the smallest normal leaves 2^(scale S) at 1)
        const float scale = fmaxf(fabsf(a.scale_log2), 1.17549435e-38f);
        const int cnt = count_of(u);
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int i = 0; i < cnt; ++i) {
            ok = wait(&B.s_full[u], (uint32_t)i, 1, true);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                // (it meets no more)
                asm volatile("bar.arrive %0, 64;\n" ::"r"(meet_id) : "memory");
                break;
            }
            tc::fence_after();
            float v[HK];
#pragma unroll
            for (int c = 0; c < HK; c += 32)
                tc::tmem_ld32(lanes + C::s_col(u) + hh * HK + c, *reinterpret_cast<uint32_t(*)[32]>(&v[c]));
            tc::tmem_ld_wait();
            const int left = a.prefix_len - (t0 + tile_of(u, i)) * KT - hh * HK;   // keys that exist
            if (left < HK) {
#pragma unroll
                for (int e = 0; e < HK; ++e) v[e] = e < left ? v[e] : -INFINITY;
            }
            float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
            for (int e = 4; e + 4 < HK; e += 8)
#pragma unroll
                for (int q = 0; q < 4; ++q) mx[q] = pf_max3(mx[q], v[e + q], v[e + 4 + q]);
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = fmax_nan(mx[q], v[HK - 4 + q]);
            // both threads of the row take the same maximum; the other's is overwritten only after
            // the products of both halves
            const float mine = fmax_nan(fmax_nan(mx[0], mx[1]), fmax_nan(mx[2], mx[3]));
            row_top[u][hh][r] = mine;
            tc::fence_before();
            meet();                              // S is read: P may overwrite it
            tc::fence_after();
            const float top = fmax_nan(mine, row_top[u][hh ^ 1][r]) * scale;
            if (i == 0) {
                m = top;
            } else if (__any_sync(0xffffffffu, !(top <= m + kPfSlack))) {
                const float mn = fmax_nan(m, top);
                const float f = m == mn ? 1.0f : sa_ex2(m - mn);
                m = mn;
                l *= f;
                // O of the earlier tiles is complete: S of this tile was issued after it.  The thread
                // of the first half rescales all of it: the product starts on that half's P
                if (hh == 0) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t w[16];
                        tc::tmem_ld16(lanes + C::o_col(u) + c, w);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * f);
                        tc::tmem_st16(lanes + C::o_col(u) + c, w);
                    }
                }
            }
            const float sub = m == -INFINITY ? 0.0f : m;
            const float2 neg = make_float2(-sub, -sub), sc2 = make_float2(scale, scale);
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
            for (int c = 0; c < HK; c += 32) {
                uint32_t w[C::kParts][16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float2 p = __ffma2_rn(make_float2(v[c + e], v[c + e + 1]), sc2, neg);
                    if (!SPLIT && (e >> 1) % 8 < kPfPoly) {
                        p = pf_exp2_poly(p);
                    } else {
                        p.x = sa_ex2(p.x);
                        p.y = sa_ex2(p.y);
                    }
                    sum[(e >> 1) & 1] = __fadd2_rn(sum[(e >> 1) & 1], p);
#pragma unroll
                    for (int part = 0; part < C::kParts; ++part) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(p.x, p.y);
                        w[part][e >> 1] = *reinterpret_cast<const uint32_t *>(&b);
                        if (part + 1 < C::kParts) {
                            const float2 back = __bfloat1622float2(b);
                            p.x -= back.x;
                            p.y -= back.y;
                        }
                    }
                }
#pragma unroll
                for (int part = 0; part < C::kParts; ++part)
                    tc::tmem_st16(lanes + C::s_col(u) + part * C::kPCols + (hh * HK + c) / 2, w[part]);
            }
            const float2 t = __fadd2_rn(sum[0], sum[1]);
            l += t.x + t.y;
            tc::tmem_st_wait();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&B.p_full[u][hh]);
        }
        // ---- the streams' results
        if (ok)
            for (int q = 0; ok && q < 2; ++q)
                if (count_of(q) > 0) ok = wait(&B.o_full[q], 0, 9, false);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) tc::fence_after();
        // The ring is free now.  Streams on the same rows: the second hands its sums over
        // (chunk-major, so that a warp's accesses are contiguous) and the first joins them.
        float4 *xo = reinterpret_cast<float4 *>(ring);                 // [D / 4][128]
        float2 *xm = reinterpret_cast<float2 *>(sQ);                   // [stream][half of the keys][128] (m, l)
        if (ok) {                                // (the queries have been read, too)
            xm[(u * 2 + hh) * 128 + r] = make_float2(m, l);
            if (pair && u == 1 && cnt > 0) {
#pragma unroll
                for (int c = hh * HD; c < hh * HD + HD; c += 16) {
                    uint32_t w[16];
                    tc::tmem_ld16(lanes + C::o_col(1) + c, w);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        xo[(c / 4 + e) * 128 + r] =
                            make_float4(__uint_as_float(w[4 * e]), __uint_as_float(w[4 * e + 1]),
                                        __uint_as_float(w[4 * e + 2]), __uint_as_float(w[4 * e + 3]));
                }
            }
        }
        asm volatile("bar.sync 9, 512;\n" ::: "memory");        // every softmax warp, whether it gave up or not
        if (!(pair && u == 1)) {
            float f0 = 1.0f, f1 = 0.0f;
            const bool both = pair && count_of(1) > 0;
            l += xm[(u * 2 + (hh ^ 1)) * 128 + r].y;
            if (both) {
                const float2 o = xm[2 * 128 + r];
                const float lo = o.y + xm[3 * 128 + r].y, mn = fmax_nan(m, o.x);
                f0 = m == mn ? 1.0f : sa_ex2(m - mn);
                f1 = o.x == mn ? 1.0f : sa_ex2(o.x - mn);
                l = l * f0 + lo * f1;
                m = mn;
            }
            const size_t at = ((size_t)split * a.c.n_kv + h) * rows;
            if (ok && hh == 0 && row < rows) *reinterpret_cast<float2 *>(a.tc_ml + (at + row) * 2) = make_float2(m, l);
            // a thread holds half a row, the stores want rows: through the warp's own 32 rows of
            // shared memory, 16-byte chunks XORed by row so that neither side conflicts
            unsigned char *stage = ring + (pair ? 128 * D * 4 : u * 128 * D * 4) + (warp & 7) * 32 * HD * 4;
            if (ok) {
#pragma unroll
                for (int c = 0; c < HD; c += 16) {
                    uint32_t w[16];
                    tc::tmem_ld16(lanes + C::o_col(u) + hh * HD + c, w);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float4 x = make_float4(__uint_as_float(w[4 * e]), __uint_as_float(w[4 * e + 1]),
                                               __uint_as_float(w[4 * e + 2]), __uint_as_float(w[4 * e + 3]));
                        if (both) {
                            const float4 y = xo[((hh * HD + c) / 4 + e) * 128 + r];
                            x.x = x.x * f0 + y.x * f1;
                            x.y = x.y * f0 + y.y * f1;
                            x.z = x.z * f0 + y.z * f1;
                            x.w = x.w * f0 + y.w * f1;
                        }
                        *reinterpret_cast<float4 *>(stage + lane * (HD * 4) + (((c / 4 + e) ^ (lane & 7)) << 4)) = x;
                    }
                }
                __syncwarp();
                constexpr int kChunks = HD / 4, kPer = 32 / kChunks;   // chunks of half a row, rows per access
                const int first = row - lane, q = lane / kChunks, c = lane % kChunks;
#pragma unroll 8
                for (int k = 0; k < 32; k += kPer) {
                    const float4 x =
                        *reinterpret_cast<const float4 *>(stage + (k + q) * (HD * 4) + ((c ^ ((k + q) & 7)) << 4));
                    if (first + k + q < rows)
                        *reinterpret_cast<float4 *>(a.tc_o + (at + first + k + q) * D + hh * HD + c * 4) = x;
                }
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// ----------------------------------------------------------------------------- host --
inline int pf_map(CUtensorMap *m, const void *base, int D, int n_kv, int keys, int box_keys) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tc::tensor_map_encoder();
    if (!enc) return CRS_ERR_CUDA;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)n_kv, (cuuint64_t)keys};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)n_kv * D * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)box_keys};
    cuuint32_t estr[3] = {1, 1, 1};
    if (enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return CRS_ERR_CUDA;
    return CRS_OK;
}

template <int D, bool SPLIT> int pf_launch(const CaArgs &a, cudaStream_t s) {
    using C = PfCfg<D, SPLIT>;
    CUtensorMap k, v;
    int e = pf_map(&k, a.pk, D, a.c.n_kv, a.prefix_len, C::kKeys);
    if (!e) e = pf_map(&v, a.pv, D, a.c.n_kv, a.prefix_len, C::kKeys);
    if (e) return e;
    CRS_TRY_CUDA(
        cudaFuncSetAttribute(cache_prefix_kernel<D, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem));
    ProfScope _ps(K_CACHE_PREFIX, s);
    cache_prefix_kernel<D, SPLIT>
        <<<(unsigned)(a.c.n_kv * a.tc_splits * a.tc_tiles), kPfThreads, C::kSmem, s>>>(a, k, v);
    CRS_CHECK_LAUNCH();
    return CRS_OK;
}

// Key splits: the grid's waves times a split's length, against the partial results that
// every split writes and the merge reads.  In microseconds, measured on one B200: a key
// tile of 128 takes about 1.5, a CTA's start and end 5, the partial results 3 TB/s.
//
// The tensor core truncates each addition to an accumulator: an f32 output, whose three
// parts of P add three times per 16 keys, is 3e-6 off after 1024 keys and 8.6e-6 after
// 2900 (a plain fp32 product over 9000 to 26000 keys 1.7e-6 to 2.9e-6).  Its splits are at
// most kPfChain keys long, and the merge adds them up with rounding.
constexpr int kPfChain = 640;
inline int pf_splits(int n_kv, int tiles, long long rows, int D, int PT, int least, int sms) {
    int best = least;
    double best_cost = 1e30;
    for (int sp = least; sp <= PT && sp <= max(least, 2 * sms); ++sp) {
        const long long ctas = (long long)n_kv * tiles * sp;
        const double waves = (double)((ctas + sms - 1) / sms);
        const double cost = waves * (((PT + sp - 1) / sp) * 1.5 + 5.0) + (double)sp * rows * n_kv * D * 8 / 3e6;
        if (cost < best_cost) {
            best_cost = cost;
            best = sp;
        }
    }
    return best;
}

}  // namespace crs
