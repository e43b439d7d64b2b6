// Decode attention over a prefix shared by the batch and each sequence's own cached
// slots, with the weights accumulated for eviction, sm_100a.
//
// The work is a list of items: (KV head, tile of query rows) over the prefix, where
// the rows are the whole batch's queries of that head, and (sequence, KV head, tile
// of its query rows) over its own slots.  An item's keys are cut into tiles; the tiles
// of all items form one sequence, of which every CTA of a fixed grid (as many as fit on
// the GPU) takes an equal share: the lengths live on the device, and ragged batches stay
// balanced without the host knowing them.  A CTA's share of an item is a piece with its
// own softmax state (m, l, unnormalised O); piece number = CTA + item, which is unique
// because one of the two grows from piece to piece.  cache_merge_kernel joins the
// pieces, divides, and turns the logits kept in the workspace into accumulated weights.
//
// The prefix of a larger batch has a pass of its own (cache_prefix.cu).
//
// Bound by memory: 537 MB of K/V (32 sequences x 8 heads x 4096 slots) take 84 us (6.4 TB/s,
// 0.99 of the measured copy rate), 268 MB of 64 sequences of 1 to 2047 slots 49 us
// (5.5 TB/s).  Three CTAs per SM with two 32 KB tiles each beat two with three (66 us
// against 74): what they hide is the start and end of an item, which count as one tile in
// the shares (without that ragged lengths took 61 us instead of 53).  The K/V copies carry
// an evict-first hint: the pieces, the prefix pass's results and the logits then stay in L2
// for the merge (15 -> 11 to 13 us).
#include <math.h>

#include "cache.cuh"

namespace crs {

constexpr int kCaWarps = 4;            // each takes 16 keys of a tile
constexpr int kCaThreads = kCaWarps * 32;
constexpr int kCaStages = 2;           // K/V tiles in the ring
constexpr int kCaRing = kCaStages + 1; // tiles whose row lists are kept
constexpr int kCaTcRows = 16;          // rows per KV head above which the prefix goes to the tensor cores
constexpr int kMgThreads = 128;
constexpr int kMgSlots = 1024;         // slots whose mass a CTA updates at a time

template <int D> constexpr int ca_tile_bytes() { return kCaKeys * D * 2; }
template <int D> constexpr int ca_scratch_bytes() { return D / 8 * 32 * 16; }
template <int D> constexpr int ca_smem_bytes() {
    return 2 * kCaStages * ca_tile_bytes<D>() + ca_scratch_bytes<D>() + kCaRing * kCaKeys * 4 + kCaRing * 2 * 8 +
           kCaWarps * 16 * 2 * 4;
}

// CTAs per SM: as many as the shared memory (76 and 38 KB) and the registers hold
template <int D> constexpr int ca_per_sm() { return D == 128 ? 3 : 5; }

// byte offset of 16-byte chunk c of row r of a tile (rows of 2 D bytes, chunks XORed by row)
template <int D> __device__ __forceinline__ int ca_off(int r, int c) { return r * (D * 2) + ((c ^ (r & 7)) << 4); }

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kCaThreads, ca_per_sm<D>()) cache_attn_kernel(CaArgs a) {
    extern __shared__ __align__(128) unsigned char ca_smem[];
    static_assert(ca_per_sm<D>() * (ca_smem_bytes<D>() + (int)sizeof(CaLens) + 1024 + 64) <= 233472, "CTAs per SM");
    constexpr int kTile = ca_tile_bytes<D>(), kChunks = D / 8, kParts = SPLIT ? 3 : 1;
    unsigned char *sK = ca_smem;                                       // [stages][64 rows][2 D bytes]
    unsigned char *sV = sK + kCaStages * kTile;
    float4 *sAcc = reinterpret_cast<float4 *>(sV + kCaStages * kTile); // [D / 8][32 lanes]
    const __nv_bfloat16 **sBase = reinterpret_cast<const __nv_bfloat16 **>(sAcc + D / 8 * 32);   // [ring][K, V]
    int *sRow = reinterpret_cast<int *>(sBase + kCaRing * 2);          // [ring][64]: token row, -1: none
    float *sM = reinterpret_cast<float *>(sRow + kCaRing * kCaKeys);   // [warps][16]
    float *sL = sM + kCaWarps * 16;
    __shared__ CaLens lens;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g_row = lane >> 2, tig = lane & 3;

    dependents_may_start();
    ca_cumulate<kCaThreads>(a, lens);
    CaCursor ahead = ca_seek(a, lens);           // next tile whose rows are listed
    CaCursor cur = ahead;                        // tile being consumed
    if (!cur.more()) {
        if (blockIdx.x == 0) wait_for_previous();
        return;
    }
    int listed = 0;

    const size_t tok_stride = (size_t)a.c.n_kv * D;
    // slots are read once per tile of 16 query rows (one tile in a step of few tokens): the
    // partial results and the logits shall stay in L2 instead
    const uint64_t once = evict_first_policy();
    // rows of the ahead tile into ring slot i % kCaRing
    auto list_tile = [&](int i) {
        if (!ahead.more()) return;
        const int slot = i % kCaRing;
        if (tid < kCaKeys) {
            const int j = ahead.t * kCaKeys + tid;
            int row = -1;
            if (ahead.prefix) {
                if (j < a.prefix_len) row = j;
            } else {
                int len, total;
                ca_lens_of(a, lens, ahead.s, len, total);
                if (j < total) row = cache_row(a.c, ahead.s, j);
            }
            sRow[slot * kCaKeys + tid] = row;
            if (tid == 0) {
                sBase[slot * 2] = (ahead.prefix ? a.pk : a.c.k) + ahead.h * D;
                sBase[slot * 2 + 1] = (ahead.prefix ? a.pv : a.c.v) + ahead.h * D;
            }
        }
        ca_advance(a, lens, ahead);
        ++listed;
    };
    // 16-byte copies of tile i's K and V rows (one commit group, empty past the last tile)
    auto load_tile = [&](int i) {
        if (i < listed) {
            const int slot = i % kCaRing, buf = i % kCaStages;
            const __nv_bfloat16 *Kb = sBase[slot * 2], *Vb = sBase[slot * 2 + 1];
#pragma unroll
            for (int e0 = 0; e0 < kCaKeys * kChunks / kCaThreads; ++e0) {
                const int e = tid + e0 * kCaThreads;
                const int r = e / kChunks, c = e % kChunks;
                const int row = sRow[slot * kCaKeys + r];
                const bool ok = row >= 0;
                const size_t off = ok ? (size_t)row * tok_stride + c * 8 : 0;
                cp_async16_zfill_once(sK + buf * kTile + ca_off<D>(r, c), Kb + off, ok, once);
                cp_async16_zfill_once(sV + buf * kTile + ca_off<D>(r, c), Vb + off, ok, once);
            }
        }
        cp_async_commit();
    };

    for (int i = 0; i < kCaStages; ++i) list_tile(i);
    __syncthreads();
    for (int i = 0; i < kCaStages - 1; ++i) load_tile(i);

    uint32_t qf[D / 16][4];
    float o[D / 8][4];
    float m_lo, m_hi, l_lo, l_hi;
    int lim_lo = 0, lim_hi = 0, lim_max = 0;
    float *log_lo = nullptr, *log_hi = nullptr;
    bool fresh = true;                           // the next tile starts a piece

    for (int i = 0; cur.more(); ++i) {
        const int buf = i % kCaStages, slot = i % kCaRing;
        if (fresh) {                             // query fragments straight from global memory
            fresh = false;
            const __nv_bfloat16 *q_lo = ca_query(a, lens, cur, g_row, &lim_lo);
            const __nv_bfloat16 *q_hi = ca_query(a, lens, cur, g_row + 8, &lim_hi);
            lim_max = __reduce_max_sync(0xffffffffu, max(lim_lo, lim_hi));
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int col = kk * 16 + e * 8 + tig * 2;
                    qf[kk][2 * e] = q_lo ? *reinterpret_cast<const uint32_t *>(q_lo + col) : 0u;
                    qf[kk][2 * e + 1] = q_hi ? *reinterpret_cast<const uint32_t *>(q_hi + col) : 0u;
                }
            }
#pragma unroll
            for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
            m_lo = m_hi = -INFINITY;
            l_lo = l_hi = 0.0f;
            log_lo = log_hi = nullptr;
            if (a.logits && !cur.prefix) {
                float *base = a.logits + ((size_t)cur.s * a.c.n_kv + cur.h) * a.M * a.ls;
                const int R = cur.rt * kCaRows + g_row;
                if (R < a.M) log_lo = base + (size_t)R * a.ls;
                if (R + 8 < a.M) log_hi = base + (size_t)(R + 8) * a.ls;
            }
        }
        cp_async_wait<kCaStages - 2>();          // tile i has landed (this thread's copies)
        __syncthreads();                         // ... everyone's; tile i - 1 is no longer read
        load_tile(i + kCaStages - 1);            // into the buffer of tile i - 1
        list_tile(i + kCaStages);                // over the rows of tile i - 1
        const int kw = warp * 16;                // this warp's 16 keys
        const int j0 = cur.t * kCaKeys + kw;
        const int *rows = sRow + slot * kCaKeys + kw;
        if (j0 < lim_max) {
            const uint32_t kb = smem_u32(sK + buf * kTile), vb = smem_u32(sV + buf * kTile);
            float s[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                // (keys 0-7, dims lo), (keys 0-7, dims hi), (keys 8-15, lo), (keys 8-15, hi)
                const int mi = lane >> 3, r = kw + (lane & 7) + ((mi >> 1) << 3), c = kk * 2 + (mi & 1);
                uint32_t b0, b1, b2, b3;
                ldsm_x4(kb + ca_off<D>(r, c), b0, b1, b2, b3);
                mma_bf16(s[0], qf[kk], b0, b1);
                mma_bf16(s[1], qf[kk], b2, b3);
            }
            float mx_lo = -INFINITY, mx_hi = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int key = nt * 8 + tig * 2 + e;
                    const bool ok = rows[key] >= 0;
                    s[nt][e] = ok && j0 + key < lim_lo ? s[nt][e] * a.scale_log2 : -INFINITY;
                    s[nt][2 + e] = ok && j0 + key < lim_hi ? s[nt][2 + e] * a.scale_log2 : -INFINITY;
                    mx_lo = fmax_nan(mx_lo, s[nt][e]);
                    mx_hi = fmax_nan(mx_hi, s[nt][2 + e]);
                }
                const int key = nt * 8 + tig * 2;
                if (log_lo) *reinterpret_cast<float2 *>(log_lo + j0 + key) = make_float2(s[nt][0], s[nt][1]);
                if (log_hi) *reinterpret_cast<float2 *>(log_hi + j0 + key) = make_float2(s[nt][2], s[nt][3]);
            }
            mx_lo = fmax_nan(mx_lo, __shfl_xor_sync(0xffffffffu, mx_lo, 1));
            mx_lo = fmax_nan(mx_lo, __shfl_xor_sync(0xffffffffu, mx_lo, 2));
            mx_hi = fmax_nan(mx_hi, __shfl_xor_sync(0xffffffffu, mx_hi, 1));
            mx_hi = fmax_nan(mx_hi, __shfl_xor_sync(0xffffffffu, mx_hi, 2));
            const float mn_lo = fmax_nan(m_lo, mx_lo), mn_hi = fmax_nan(m_hi, mx_hi);   // a NaN logit stays one
            const float c_lo = (mn_lo == -INFINITY) ? 1.0f : sa_ex2(m_lo - mn_lo);
            const float c_hi = (mn_hi == -INFINITY) ? 1.0f : sa_ex2(m_hi - mn_hi);
            float ps_lo = 0.0f, ps_hi = 0.0f;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    s[nt][e] = (s[nt][e] == -INFINITY) ? 0.0f : sa_ex2(s[nt][e] - mn_lo);
                    s[nt][2 + e] = (s[nt][2 + e] == -INFINITY) ? 0.0f : sa_ex2(s[nt][2 + e] - mn_hi);
                    ps_lo += s[nt][e];
                    ps_hi += s[nt][2 + e];
                }
            }
            l_lo = l_lo * c_lo + ps_lo;
            l_hi = l_hi * c_hi + ps_hi;
            m_lo = mn_lo;
            m_hi = mn_hi;
            if (c_lo != 1.0f || c_hi != 1.0f) {
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    o[j][0] *= c_lo; o[j][1] *= c_lo;
                    o[j][2] *= c_hi; o[j][3] *= c_hi;
                }
            }
            // f32 output: P as three bf16 parts (24 bits); bf16 output: P rounded once, half a bf16
            // step, as the output itself is
            uint32_t pa[kParts][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float x = s[q >> 1][(q & 1) * 2], y = s[q >> 1][(q & 1) * 2 + 1];
#pragma unroll
                for (int part = 0; part < kParts; ++part) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
                    pa[part][q] = *reinterpret_cast<const uint32_t *>(&h);
                    const float2 back = __bfloat1622float2(h);
                    x -= back.x;
                    y -= back.y;
                }
            }
#pragma unroll
            for (int jj = 0; jj < D / 16; ++jj) {
                // (keys 0-7, dims 16jj..), (keys 8-15, dims 16jj..), (keys 0-7, 16jj+8..), (keys 8-15, 16jj+8..)
                const int mi = lane >> 3, r = kw + (lane & 7) + ((mi & 1) << 3), c = jj * 2 + (mi >> 1);
                uint32_t b0, b1, b2, b3;
                ldsm_x4_t(vb + ca_off<D>(r, c), b0, b1, b2, b3);
                if constexpr (SPLIT) {
                    // the tensor core truncates what it adds to: short chains, joined with rounding
                    float t[2][4] = {};
#pragma unroll
                    for (int part = kParts - 1; part >= 0; --part) {
                        mma_bf16(t[0], pa[part], b0, b1);
                        mma_bf16(t[1], pa[part], b2, b3);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[2 * jj][e] += t[0][e];
                        o[2 * jj + 1][e] += t[1][e];
                    }
                } else {
                    mma_bf16(o[2 * jj], pa[0], b0, b1);
                    mma_bf16(o[2 * jj + 1], pa[0], b2, b3);
                }
            }
        } else if (a.logits && !cur.prefix) {
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const int key = nt * 8 + tig * 2;
                if (log_lo) *reinterpret_cast<float2 *>(log_lo + j0 + key) = make_float2(-INFINITY, -INFINITY);
                if (log_hi) *reinterpret_cast<float2 *>(log_hi + j0 + key) = make_float2(-INFINITY, -INFINITY);
            }
        }

        // ---- end of the piece: the warps' states are joined in warp order through 16 D floats
        if (cur.ends()) {
            fresh = true;
            l_lo += __shfl_xor_sync(0xffffffffu, l_lo, 1);
            l_lo += __shfl_xor_sync(0xffffffffu, l_lo, 2);
            l_hi += __shfl_xor_sync(0xffffffffu, l_hi, 1);
            l_hi += __shfl_xor_sync(0xffffffffu, l_hi, 2);
            if (tig == 0) {
                sM[warp * 16 + g_row] = m_lo;
                sM[warp * 16 + g_row + 8] = m_hi;
                sL[warp * 16 + g_row] = l_lo;
                sL[warp * 16 + g_row + 8] = l_hi;
            }
            __syncthreads();
            float M_lo = -INFINITY, M_hi = -INFINITY;
#pragma unroll
            for (int v = 0; v < kCaWarps; ++v) {
                M_lo = fmax_nan(M_lo, sM[v * 16 + g_row]);
                M_hi = fmax_nan(M_hi, sM[v * 16 + g_row + 8]);
            }
            const float f_lo = m_lo == -INFINITY ? 0.0f : sa_ex2(m_lo - M_lo);
            const float f_hi = m_hi == -INFINITY ? 0.0f : sa_ex2(m_hi - M_hi);
#pragma unroll
            for (int v = kCaWarps - 1; v >= 0; --v) {
                if (warp == v) {
#pragma unroll
                    for (int j = 0; j < D / 8; ++j) {
                        float4 x = make_float4(o[j][0] * f_lo, o[j][1] * f_lo, o[j][2] * f_hi, o[j][3] * f_hi);
                        if (v < kCaWarps - 1) {
                            const float4 y = sAcc[j * 32 + lane];
                            x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
                        }
                        if (v > 0) {
                            sAcc[j * 32 + lane] = x;
                        } else {
                            o[j][0] = x.x; o[j][1] = x.y; o[j][2] = x.z; o[j][3] = x.w;
                        }
                    }
                }
                if (v > 0) __syncthreads();
            }
            if (warp == 0) {
                const size_t piece = (size_t)(blockIdx.x + ca_item(a, cur));
                float *po = a.part_o + piece * (kCaRows * D);
                float *pm = a.part_ml + piece * (kCaRows * 2);
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    const int col = j * 8 + tig * 2;
                    if (lim_lo > 0) *reinterpret_cast<float2 *>(po + g_row * D + col) = make_float2(o[j][0], o[j][1]);
                    if (lim_hi > 0)
                        *reinterpret_cast<float2 *>(po + (g_row + 8) * D + col) = make_float2(o[j][2], o[j][3]);
                }
                if (lane < kCaRows) {
                    float Mx = -INFINITY, L = 0.0f;
#pragma unroll
                    for (int v = 0; v < kCaWarps; ++v) Mx = fmax_nan(Mx, sM[v * 16 + lane]);
#pragma unroll
                    for (int v = 0; v < kCaWarps; ++v)
                        if (sM[v * 16 + lane] != -INFINITY) L += sL[v * 16 + lane] * sa_ex2(sM[v * 16 + lane] - Mx);
                    *reinterpret_cast<float2 *>(pm + lane * 2) = make_float2(Mx, L);
                }
            }
            __syncthreads();                     // sM, sL and sAcc are reused
        }
        ca_advance(a, lens, cur);
    }
    cp_async_wait<0>();
    // The merge waits for this kernel, so one CTA of it waits for the prefix pass (all of them
    // would keep their places on SMs that the prefix pass leaves free).
    if (blockIdx.x == 0) wait_for_previous();
}

// --------------------------------------------------------------------------- merge --
// A row's pieces: first those of its own item, then the prefix's.
struct MgRow {
    long long own0, pre0;      // first piece number
    int n_own, n_pre;
    int r_own, r_pre;          // row within the pieces' 16
    int h;
    long long r_tc;            // row of the tensor-core prefix pass
};
__device__ __forceinline__ MgRow mg_row(const CaArgs &a, int s, int h, int R, int before, int T, long long w) {
    MgRow m;
    const long long P = ca_prefix_units(a);
    m.n_own = m.n_pre = 0;
    m.own0 = m.pre0 = 0;
    m.h = h;
    const int rt = R / kCaRows;
    m.r_own = R - rt * kCaRows;
    if (T > 0) {
        const long long x = ((long long)s * a.c.n_kv + h) * a.RT + rt;
        const long long first = P + (long long)before * a.c.n_kv * a.RT +
                                ((long long)h * a.RT + rt) * (T + kItemCost) + kItemCost;
        const long long c0 = ca_div(first, w), c1 = ca_div(first + T - 1, w);
        m.own0 = c0 + (long long)a.c.n_kv * a.PRT + x;
        m.n_own = (int)(c1 - c0 + 1);
    }
    const long long Rg = (long long)s * a.M + R;
    m.r_tc = Rg;
    if (a.PT > 0) {
        const int prt = (int)(Rg / kCaRows);
        m.r_pre = (int)(Rg - (long long)prt * kCaRows);
        const long long x = (long long)h * a.PRT + prt, first = x * ca_units(a.PT) + kItemCost;
        const long long c0 = ca_div(first, w), c1 = ca_div(first + a.PT - 1, w);
        m.pre0 = c0 + x;
        m.n_pre = (int)(c1 - c0 + 1);
    } else {
        m.r_pre = 0;
        m.n_pre = a.tc_splits;
    }
    return m;
}
// Piece p of the row: index of its (m, l) pair, and of its D floats, in the arrays of the
// slots' pass (tc false) or of the prefix pass.
__device__ __forceinline__ size_t mg_piece(const CaArgs &a, const MgRow &m, int p, bool &tc) {
    tc = false;
    if (p < m.n_own) return (size_t)(m.own0 + p) * kCaRows + m.r_own;
    if (a.PT > 0) return (size_t)(m.pre0 + p - m.n_own) * kCaRows + m.r_pre;
    tc = true;
    return ((size_t)(p - m.n_own) * a.c.n_kv + m.h) * ((size_t)a.c.n_seq * a.M) + (size_t)m.r_tc;
}

// Largest m and total l of the row's pieces, for LANES neighbouring lanes of a warp each
// (all of its lanes take part; -inf and 0 when there is nothing).
template <int LANES>
__device__ __forceinline__ float2 mg_stat(const CaArgs &a, const MgRow &m, int lane) {
    const int n = m.n_own + m.n_pre;
    float mx = -INFINITY, l = 0.0f;
#pragma unroll 4
    for (int p = lane % LANES; p < n; p += LANES) {
        bool tc;
        const size_t k = mg_piece(a, m, p, tc);
        const float2 v = *reinterpret_cast<const float2 *>((tc ? a.tc_ml : a.part_ml) + k * 2);
        const float mn = fmax_nan(mx, v.x);
        if (mn == -INFINITY) continue;
        l = l * exp2f(mx - mn) + v.y * exp2f(v.x - mn);
        mx = mn;
    }
    float Mx = mx;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) Mx = fmax_nan(Mx, __shfl_xor_sync(0xffffffffu, Mx, o));
    l = mx == -INFINITY ? 0.0f : l * exp2f(mx - Mx);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    return make_float2(Mx, l);
}

// The CTAs of one (sequence, KV head): `joins` join the pieces of its rows, WPR warps to a
// row, the others update every chunks-th run of kMgSlots slots' mass.  The two kinds run
// side by side: a row's statistics are found again where they are needed, which is less
// than waiting for them.
template <int D, int WPR, typename OutT>
__global__ void __launch_bounds__(kMgThreads, 8) cache_merge_kernel(CaArgs a, int joins, int chunks) {
    constexpr int kE = D / 32, kRows = kMgThreads / 32 / WPR;
    extern __shared__ float mg_z[];              // mass: [M] lse in log2 units
    __shared__ float red[WPR > 1 ? kMgThreads / 32 : 1][D];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int sh = blockIdx.x / (joins + chunks), part = blockIdx.x - sh * (joins + chunks);
    const int s = sh / a.c.n_kv, h = sh - s * a.c.n_kv;
    wait_for_previous();
    const int len = cache_len(a.c, s), n = cache_new(a.c, a.n_new, a.n_tok, s, len);
    const int total = len + n, rows = n * a.G;
    if (part >= joins && (part - joins) * kMgSlots >= total) return;
    const int before = a.cum[s], after = a.cum[s + 1], all = a.cum[a.c.n_seq];
    const int T = after > before ? after - before - kItemCost : 0;
    const long long w = ca_share(a, ca_prefix_units(a) + (long long)all * a.c.n_kv * a.RT);

    if (part < joins) {
        const int R = part * kRows + warp / WPR, sub = warp % WPR;
        float acc[kE];
#pragma unroll
        for (int e = 0; e < kE; ++e) acc[e] = 0.0f;
        float2 st = make_float2(-INFINITY, 0.0f);
        if (R < rows) {
            const MgRow m = mg_row(a, s, h, R, before, T, w);
            st = mg_stat<32>(a, m, lane);
            const int np = m.n_own + m.n_pre;
            if (st.x != -INFINITY) {
                // lane q knows the address and the weight of the warp's q-th piece
                for (int p0 = sub; p0 < np; p0 += 32 * WPR) {
                    const int p = p0 + lane * WPR, count = min(32, (np - p0 + WPR - 1) / WPR);
                    const float *src = nullptr;
                    float f = 0.0f;
                    if (p < np) {
                        bool tc;
                        const size_t k = mg_piece(a, m, p, tc);
                        const float pm = (tc ? a.tc_ml : a.part_ml)[k * 2];
                        src = (tc ? a.tc_o : a.part_o) + k * D;
                        f = pm == -INFINITY ? 0.0f : exp2f(pm - st.x);
                    }
#pragma unroll 8
                    for (int q = 0; q < count; ++q) {
                        const float *from = reinterpret_cast<const float *>(
                            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), q));
                        const float fq = __shfl_sync(0xffffffffu, f, q);
                        // a piece whose rows all saw nothing may hold anything: weight 0, not added
                        if constexpr (kE == 4) {
                            const float4 v = *reinterpret_cast<const float4 *>(from + lane * 4);
                            if (fq != 0.0f) {
                                acc[0] += fq * v.x; acc[1] += fq * v.y; acc[2] += fq * v.z; acc[3] += fq * v.w;
                            }
                        } else {
                            const float2 v = *reinterpret_cast<const float2 *>(from + lane * 2);
                            if (fq != 0.0f) {
                                acc[0] += fq * v.x; acc[1] += fq * v.y;
                            }
                        }
                    }
                }
            }
        }
        if constexpr (WPR > 1) {
#pragma unroll
            for (int e = 0; e < kE; ++e) red[warp][lane * kE + e] = acc[e];
            __syncthreads();
            if (sub == 0) {
#pragma unroll
                for (int v = 1; v < WPR; ++v)
#pragma unroll
                    for (int e = 0; e < kE; ++e) acc[e] += red[warp + v][lane * kE + e];
            }
        }
        if (R < a.M && sub == 0) {
            const int i = R / a.G, g = R - i * a.G;
            const size_t row = ((size_t)s * a.n_tok + i) * a.n_q + h * a.G + g;
            OutT *dst = static_cast<OutT *>(a.O) + row * D + lane * kE;
            // nothing seen: zeros; a NaN or infinite sum passes through
            const float L = st.y, f = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
            for (int e = 0; e < kE; e += 2) {
                const float x = L == 0.0f ? 0.0f : acc[e] * f, y = L == 0.0f ? 0.0f : acc[e + 1] * f;
                if constexpr (sizeof(OutT) == 4) *reinterpret_cast<float2 *>(dst + e) = make_float2(x, y);
                else *reinterpret_cast<__nv_bfloat162 *>(dst + e) = __floats2bfloat162_rn(x, y);
            }
            if (a.lse && lane == 0) a.lse[row] = L == 0.0f ? -INFINITY : (st.x + log2f(L)) * 0.6931471805599453f;
        }
        return;
    }

    // ---- mass: sum over the rows of 2^(logit - lse); a row that sees nothing adds 0
    for (int R0 = 0; R0 < rows; R0 += kMgThreads / 8) {          // eight lanes to a row
        const int R = R0 + tid / 8;
        MgRow m = mg_row(a, s, h, min(R, rows - 1), before, T, w);
        const float2 st = mg_stat<8>(a, m, lane);
        if (tid % 8 == 0 && R < rows) mg_z[R] = st.y != 0.0f ? st.x + log2f(st.y) : INFINITY;
    }
    __syncthreads();
    const float *lg = a.logits + (size_t)sh * a.M * a.ls;
    constexpr int kPairs = kMgSlots / (2 * kMgThreads);          // pairs of slots per thread
    for (int j0 = (part - joins) * kMgSlots + tid * 2; j0 - tid * 2 < total; j0 += chunks * kMgSlots) {
        float2 sum[kPairs], old[kPairs];
        const size_t at = (size_t)sh * a.c.cap;
#pragma unroll
        for (int q = 0; q < kPairs; ++q) {
            const int j = j0 + q * 2 * kMgThreads;
            sum[q] = make_float2(0.0f, 0.0f);
            old[q].x = j < total ? a.c.mass[at + j] : 0.0f;
            old[q].y = j + 1 < total ? a.c.mass[at + j + 1] : 0.0f;
        }
#pragma unroll 2
        for (int R = 0; R < rows; ++R) {
            const float z = mg_z[R];
#pragma unroll
            for (int q = 0; q < kPairs; ++q) {
                const int j = j0 + q * 2 * kMgThreads;
                if (j >= total) continue;
                const float2 v = *reinterpret_cast<const float2 *>(lg + (size_t)R * a.ls + j);
                sum[q].x += exp2f(v.x - z);
                sum[q].y += exp2f(v.y - z);
            }
        }
#pragma unroll
        for (int q = 0; q < kPairs; ++q) {
            const int j = j0 + q * 2 * kMgThreads;
            if (j < total) a.mass_out[at + j] = a.decay * old[q].x + sum[q].x;
            if (j + 1 < total) a.mass_out[at + j + 1] = a.decay * old[q].y + sum[q].y;
        }
    }
}

// ----------------------------------------------------------------------------- host --
struct CaPlan {
    int grid, PT, PRT, RT, M, tc_splits, tc_tiles;
    size_t part_o, part_ml, tc_o, tc_ml, cum, logits, total;   // workspace offsets
    int ls;
};

static int ca_validate(const crs_cache_attn_params *p) {
    if (!p) return CRS_ERR_INVALID_ARG;
    const int st = cache_validate(&p->c);
    if (st) return st;
    if (p->n_q < 1 || p->n_tok < 1 || p->prefix_len < 0) return CRS_ERR_INVALID_ARG;
    if (p->out_dtype != CRS_F32 && p->out_dtype != CRS_BF16) return CRS_ERR_INVALID_ARG;
    if (p->n_q % p->c.n_kv != 0 || p->n_q / p->c.n_kv > 64) return CRS_ERR_UNSUPPORTED;
    if ((long long)p->n_tok * (p->n_q / p->c.n_kv) > 1024) return CRS_ERR_UNSUPPORTED;
    if (p->prefix_len > 0x7fffffff - 1024 || p->c.cap > 0x7fffffff - 1024) return CRS_ERR_UNSUPPORTED;
    if ((long long)p->c.n_seq * p->n_tok * p->n_q > 0x3fffffffLL) return CRS_ERR_UNSUPPORTED;
    // the units of one KV head's sequences are counted in 32 bits
    if ((long long)p->c.n_seq * (p->c.cap / kCaKeys + 2) > 0x7fffffffLL) return CRS_ERR_UNSUPPORTED;
    return CRS_OK;
}

static CaPlan ca_plan(const crs_cache_attn_params *p) {
    CaPlan q;
    const int G = p->n_q / p->c.n_kv, D = p->c.D;
    q.M = p->n_tok * G;
    q.RT = ceil_div(q.M, kCaRows);
    q.grid = cache_sms() * (D == 128 ? ca_per_sm<128>() : ca_per_sm<64>());
    // the tensor-core pass pays off once the batch's rows exceed a tile or two of the plain one
    const long long rows = (long long)p->c.n_seq * q.M;
    const bool tc = p->prefix_len > 0 && rows > kCaTcRows;
    q.tc_tiles = (int)ceil_div_ll(rows, kPfRows);
    q.tc_splits = tc ? pf_splits(p->c.n_kv, q.tc_tiles, rows, D,
                                 ceil_div(p->prefix_len, p->out_dtype == CRS_F32 ? 64 : 128),
                                 p->out_dtype == CRS_F32 ? ceil_div(p->prefix_len, kPfChain) : 1, cache_sms())
                     : 0;
    q.PT = tc ? 0 : ceil_div(p->prefix_len, kCaKeys);
    q.PRT = q.PT > 0 ? ceil_div(p->c.n_seq * q.M, kCaRows) : 0;
    const size_t items = (size_t)p->c.n_kv * q.PRT + (size_t)p->c.n_seq * p->c.n_kv * q.RT;
    const size_t pieces = items + q.grid;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    size_t at = 0;
    q.part_o = at;
    at += up(pieces * kCaRows * D * 4);
    q.part_ml = at;
    at += up(pieces * kCaRows * 2 * 4);
    const size_t parts = (size_t)q.tc_splits * p->c.n_kv * p->c.n_seq * q.M;
    q.tc_o = at;
    at += up(parts * D * 4);
    q.tc_ml = at;
    at += up(parts * 2 * 4);
    q.cum = at;
    at += up(((size_t)p->c.n_seq + 1) * 4);
    q.ls = ceil_div(p->c.cap, kCaKeys) * kCaKeys;
    q.logits = at;
    if (p->want_mass) at += up((size_t)p->c.n_seq * p->c.n_kv * q.M * q.ls * 4);
    q.total = at;
    return q;
}

template <int D, bool SPLIT> int ca_launch(const CaArgs &a, cudaStream_t s) {
    const int smem = ca_smem_bytes<D>();
    CRS_TRY_CUDA(
        cudaFuncSetAttribute(cache_attn_kernel<D, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    ProfScope _ps(K_CACHE_ATTN, s);
    CRS_TRY_CUDA(launch_chained(cache_attn_kernel<D, SPLIT>, (unsigned)a.grid, kCaThreads, smem, s, a.tc_splits > 0, a));
    return CRS_OK;
}

template <int D, int WPR, typename OutT> int mg_launch_rows(const CaArgs &a, cudaStream_t s) {
    const long long sh = (long long)a.c.n_seq * a.c.n_kv;
    const int joins = ceil_div(a.M * WPR, kMgThreads / 32);
    // the mass of up to two waves of CTAs (eight fit on an SM), more slots to a CTA beyond that
    const long long most = max(1LL, (long long)cache_sms() * 16 / sh);
    const int chunks = a.logits ? (int)min(most, (long long)ceil_div(a.c.cap, kMgSlots)) : 0;
    const long long ctas = sh * (joins + chunks);
    if (ctas > 0x7fffffffLL) return CRS_ERR_UNSUPPORTED;
    ProfScope _ps(K_CACHE_MERGE, s);
    CRS_TRY_CUDA(launch_chained(cache_merge_kernel<D, WPR, OutT>, (unsigned)ctas, kMgThreads, (size_t)a.M * 4, s, true, a,
                                joins, chunks));
    return CRS_OK;
}
template <int D, typename OutT> int mg_launch(const CaArgs &a, cudaStream_t s) {
    // one warp per row while the rows fill the GPU, else four share a row's pieces
    const long long rows = (long long)a.c.n_seq * a.c.n_kv * a.M;
    return rows >= (long long)cache_sms() * 8 ? mg_launch_rows<D, 1, OutT>(a, s) : mg_launch_rows<D, 4, OutT>(a, s);
}

}  // namespace crs

using namespace crs;

extern "C" size_t crs_cache_attn_workspace_size(const crs_cache_attn_params *p) {
    if (ca_validate(p)) return 0;
    return ca_plan(p).total;
}

extern "C" int crs_cache_attn(const crs_cache_attn_params *p, const crs_cache_state *st, const void *Q,
                              const int32_t *n_new, const void *prefix_k, const void *prefix_v, void *O, float *lse,
                              float *mass_out, void *ws, size_t ws_bytes, void *stream) {
    int e = ca_validate(p);
    if (e) return e;
    if ((e = cache_check_state(st))) return e;
    if (!Q || !O || (p->prefix_len > 0 && (!prefix_k || !prefix_v))) return CRS_ERR_INVALID_ARG;
    if (p->want_mass && (!mass_out || !st->mass)) return CRS_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(prefix_k) |
         reinterpret_cast<uintptr_t>(prefix_v) | reinterpret_cast<uintptr_t>(O) | reinterpret_cast<uintptr_t>(ws)) & 15)
        return CRS_ERR_INVALID_ARG;
    const CaPlan q = ca_plan(p);
    if (!ws || ws_bytes < q.total) return CRS_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned char *w = static_cast<unsigned char *>(ws);
    CaArgs a;
    a.c = cache_dev(&p->c, st);
    a.Q = static_cast<const __nv_bfloat16 *>(Q);
    a.pk = static_cast<const __nv_bfloat16 *>(prefix_k);
    a.pv = static_cast<const __nv_bfloat16 *>(prefix_v);
    a.n_new = n_new;
    a.n_q = p->n_q;
    a.G = p->n_q / p->c.n_kv;
    a.n_tok = p->n_tok;
    a.M = q.M;
    a.RT = q.RT;
    a.prefix_len = p->prefix_len;
    a.PT = q.PT;
    a.PRT = q.PRT;
    a.grid = q.grid;
    a.tc_splits = q.tc_splits;
    a.tc_tiles = q.tc_tiles;
    a.scale_log2 = p->scale * kLog2e;
    a.decay = p->decay;
    a.part_o = reinterpret_cast<float *>(w + q.part_o);
    a.part_ml = reinterpret_cast<float *>(w + q.part_ml);
    a.tc_o = reinterpret_cast<float *>(w + q.tc_o);
    a.tc_ml = reinterpret_cast<float *>(w + q.tc_ml);
    a.cum = reinterpret_cast<int *>(w + q.cum);
    a.logits = p->want_mass ? reinterpret_cast<float *>(w + q.logits) : nullptr;
    a.ls = q.ls;
    a.O = O;
    a.lse = lse;
    a.mass_out = mass_out;
    const bool f32 = p->out_dtype == CRS_F32;
    if (a.tc_splits > 0) {
        if (p->c.D == 128) e = f32 ? pf_launch<128, true>(a, s) : pf_launch<128, false>(a, s);
        else e = f32 ? pf_launch<64, true>(a, s) : pf_launch<64, false>(a, s);
        if (e) return e;
    }
    if (p->c.D == 128) e = f32 ? ca_launch<128, true>(a, s) : ca_launch<128, false>(a, s);
    else e = f32 ? ca_launch<64, true>(a, s) : ca_launch<64, false>(a, s);
    if (e) return e;
    if (p->c.D == 128) return f32 ? mg_launch<128, float>(a, s) : mg_launch<128, __nv_bfloat16>(a, s);
    return f32 ? mg_launch<64, float>(a, s) : mg_launch<64, __nv_bfloat16>(a, s);
}
