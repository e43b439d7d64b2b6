// What the kernels of the paged decode cache share: its state on the device, slot
// addresses, and the host checks (sm_100a).
#pragma once

#include <atomic>

#include "common.cuh"

namespace crs {

struct CacheDev {
    __nv_bfloat16 *k, *v;
    const int32_t *table;
    int32_t *pos;
    float *mass;
    int32_t *seq_len, *next_pos;
    int n_seq, n_kv, D, page_size, max_pages, n_pages, cap;
};

inline CacheDev cache_dev(const crs_cache_params *p, const crs_cache_state *st) {
    CacheDev c;
    c.k = static_cast<__nv_bfloat16 *>(st->k_pool);
    c.v = static_cast<__nv_bfloat16 *>(st->v_pool);
    c.table = st->block_table;
    c.pos = st->pos;
    c.mass = st->mass;
    c.seq_len = st->seq_len;
    c.next_pos = st->next_pos;
    c.n_seq = p->n_seq;
    c.n_kv = p->n_kv;
    c.D = p->D;
    c.page_size = p->page_size;
    c.max_pages = p->max_pages;
    c.n_pages = p->n_pages;
    c.cap = p->cap;
    return c;
}

// Row of slot j (0 <= j < cap) in the pools' token dimension; -1 (flagged) when its
// block table entry is outside the pool.
__device__ __forceinline__ int cache_row(const CacheDev &c, int s, int j) {
    const int lp = j / c.page_size;
    const int page = __ldg(c.table + (size_t)s * c.max_pages + lp);
    if ((unsigned)page >= (unsigned)c.n_pages) {
        raise_error(CRS_DEVERR_INDEX);
        return -1;
    }
    return page * c.page_size + (j - lp * c.page_size);
}

// Slots in use before this step's tokens, and the new tokens that count.
__device__ __forceinline__ int cache_len(const CacheDev &c, int s) { return min(max(c.seq_len[s], 0), c.cap); }
__device__ __forceinline__ int cache_new(const CacheDev &c, const int32_t *n_new, int n_tok, int s, int len) {
    const int n = n_new ? min(max(n_new[s], 0), n_tok) : n_tok;
    return min(n, c.cap - len);
}

inline int cache_validate(const crs_cache_params *p) {
    if (!p) return CRS_ERR_INVALID_ARG;
    if (p->n_seq < 1 || p->n_kv < 1 || p->page_size < 1 || p->max_pages < 1 || p->n_pages < 1 || p->cap < 1)
        return CRS_ERR_INVALID_ARG;
    if (p->D != 64 && p->D != 128) return CRS_ERR_UNSUPPORTED;
    if (p->n_seq > 4096 || p->n_kv > 4096) return CRS_ERR_UNSUPPORTED;
    if ((long long)p->max_pages * p->page_size < p->cap) return CRS_ERR_UNSUPPORTED;
    if ((long long)p->n_pages * p->page_size > 0x7fffffffLL) return CRS_ERR_UNSUPPORTED;
    return CRS_OK;
}
inline int cache_check_state(const crs_cache_state *st) {
    if (!st || !st->k_pool || !st->v_pool || !st->block_table || !st->seq_len || !st->next_pos)
        return CRS_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(st->k_pool) | reinterpret_cast<uintptr_t>(st->v_pool)) & 15)
        return CRS_ERR_INVALID_ARG;
    return CRS_OK;
}

// SM count of the current device, looked up once per device (148 where it cannot be
// read: the sizing stays valid).
inline int cache_sms() {
    static std::atomic<int> known[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 148;
    }
    if (dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
        cudaGetLastError();
        return 148;
    }
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

constexpr int kCaRows = 16;            // query rows of an item (M of mma.sync)
constexpr int kCaKeys = 64;            // keys per tile

// Programmatic dependent launch: the next kernel of the chain may start once every CTA of
// this one has said so, and waits for the end of this one where it needs its results.
// Without the launch attribute both do nothing.
__device__ __forceinline__ void dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t launch_chained(void (*kernel)(Params...), unsigned grid, int threads, size_t smem, cudaStream_t s, bool chained,
                           Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = chained ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// What the attention kernels and the merge of their partial results are given.
struct CaArgs {
    CacheDev c;
    const __nv_bfloat16 *Q, *pk, *pv;
    const int32_t *n_new;
    int n_q, G, n_tok;
    int M;             // query rows of one (sequence, KV head): n_tok * G
    int RT;            // row tiles of an own item
    int prefix_len;
    int PT;            // key tiles of a prefix item (0: the prefix has a pass of its own)
    int PRT;           // its row tiles, over n_seq * M rows
    int grid;          // CTAs that share the tile sequence
    int tc_splits;     // key splits of cache_prefix_kernel (0: not launched)
    int tc_tiles;      // its row tiles per KV head, kPfRows rows each
    float scale_log2, decay;
    float *part_o, *part_ml;       // pieces: [piece][16][D], [piece][16][2] (m in log2 units, l)
    float *tc_o, *tc_ml;           // [split][KV head][n_seq * M][D], [..][2]
    int *cum;                      // [n_seq + 1] units of the sequences before each
    float *logits;                 // [sequence][KV head][M][ls] log2-scaled, or null
    int ls;
    void *O;
    float *lse, *mass_out;
};


// The work of the batch in units.  An item of T key tiles counts T + kItemCost units, the
// first of them for its start and end (query rows, first maximum, result), which cost
// about what a tile does; the items' units follow one another and CTA c of the grid has
// [c w, (c + 1) w).  Tile t of an item that starts at unit x is unit x + kItemCost + t.
constexpr int kItemCost = 1;

__device__ __forceinline__ int ca_units(int tiles) { return tiles > 0 ? tiles + kItemCost : 0; }
__device__ __forceinline__ long long ca_prefix_units(const CaArgs &a) {
    return (long long)a.c.n_kv * a.PRT * ca_units(a.PT);
}
// n / d of numbers >= 0, with the short division where both fit
__device__ __forceinline__ long long ca_div(long long n, long long d) {
    return ((n | d) >> 32) == 0 ? (long long)((uint32_t)n / (uint32_t)d) : n / d;
}
__device__ __forceinline__ long long ca_share(const CaArgs &a, long long W) {
    return W > a.grid ? ca_div(W + a.grid - 1, a.grid) : 1;
}

// What a CTA keeps of the sequences' lengths, in shared memory: where its share starts, and
// the slots in use before and with the new tokens of the kLensKept sequences from there
// (all of a batch that has no more; others are read again where they are needed).
constexpr int kLensKept = 128;
struct CaLens {
    long long units;               // of the whole batch (prefix items aside: per KV head and row tile)
    int start;                     // the sequence that the CTA's share of the own items starts in
    int before;                    // units of the sequences before it
    int first;                     // the first one kept
    int scan[8];
    int len[kLensKept], tot[kLensKept];
};
__device__ __forceinline__ void ca_lens_of(const CaArgs &a, const CaLens &L, int s, int &len, int &total) {
    const int k = s - L.first;
    if ((unsigned)k < (unsigned)kLensKept) {
        len = L.len[k];
        total = L.tot[k];
    } else {
        len = cache_len(a.c, s);
        total = len + cache_new(a.c, a.n_new, a.n_tok, s, len);
    }
}
// key tiles of a sequence's own items (none without a token to ask)
__device__ __forceinline__ int ca_tiles(int len, int total) {
    return total > len ? (total + kCaKeys - 1) / kCaKeys : 0;
}
__device__ __forceinline__ int ca_tiles_of(const CaArgs &a, const CaLens &L, int s) {
    int len, total;
    ca_lens_of(a, L, s, len, total);
    return ca_tiles(len, total);
}

// Fills it (one block; barriers inside).  CTA 0 leaves the units of the sequences before
// each one in a.cum for the merge.
template <int THREADS> __device__ __forceinline__ void ca_cumulate(const CaArgs &a, CaLens &L) {
    const int n = a.c.n_seq, per = (n + THREADS - 1) / THREADS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int s0 = min(n, tid * per), s1 = min(n, s0 + per);
    auto units_of = [&](int s) {
        const int len = cache_len(a.c, s);
        return ca_units(ca_tiles(len, len + cache_new(a.c, a.n_new, a.n_tok, s, len)));
    };
    static_assert(THREADS >= kLensKept, "a thread per kept sequence");
    const bool all_kept = n <= kLensKept;
    int sum = 0;
    if (all_kept) {
        if (tid < n) {
            const int len = cache_len(a.c, tid), total = len + cache_new(a.c, a.n_new, a.n_tok, tid, len);
            L.len[tid] = len;
            L.tot[tid] = total;
            sum = ca_units(ca_tiles(len, total));
        }
    } else {
#pragma unroll 4
        for (int s = s0; s < s1; ++s) sum += units_of(s);
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) L.scan[warp] = inc;
    if (tid == 0) {
        L.start = n;
        L.first = 0;
        L.before = 0;
    }
    __syncthreads();
    int base = inc - sum, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) base += L.scan[w];
        all += L.scan[w];
    }
    const long long P = ca_prefix_units(a), K = (long long)a.c.n_kv * a.RT;
    const long long n0 = max(0LL, blockIdx.x * ca_share(a, P + all * K) - P);      // of the own items
    if (tid == 0) L.units = all;
    const bool here = base * K <= n0 && n0 < (long long)(base + sum) * K;
    if (all_kept) {
        if (here) {
            L.start = tid;
            L.before = base;
        }
        if (blockIdx.x == 0 && tid < n) a.cum[tid + 1] = base + sum;
        if (blockIdx.x == 0 && tid == 0) a.cum[0] = 0;
        __syncthreads();
        return;
    }
    if (here) {
        int b = base;
        for (int s = s0; s < s1; ++s) {
            const int u = units_of(s);
            if (n0 < (long long)(b + u) * K) {
                L.start = L.first = s;
                L.before = b;
                break;
            }
            b += u;
        }
    }
    if (blockIdx.x == 0) {
        if (tid == 0) a.cum[0] = 0;
        int b = base;
        for (int s = s0; s < s1; ++s) {
            b += units_of(s);
            a.cum[s + 1] = b;
        }
    }
    __syncthreads();
    const int s = L.first + tid;
    if (tid < kLensKept && s < n) {
        const int len = cache_len(a.c, s);
        L.len[tid] = len;
        L.tot[tid] = len + cache_new(a.c, a.n_new, a.n_tok, s, len);
    }
    __syncthreads();
}

// A tile in the sequence of a CTA's tiles.
struct CaCursor {
    bool prefix;
    int s, h, rt;                  // own: sequence, KV head, row tile; prefix: h, rt
    int t, T;                      // tile of the item, tiles of the item
    long long unit, stop;          // the tile's unit; the CTA's share ends before unit stop
    __device__ __forceinline__ bool more() const { return unit < stop; }
    // the last tile of the item, or of the CTA's share of it
    __device__ __forceinline__ bool ends() const { return t == T - 1 || unit == stop - 1; }
};

__device__ __forceinline__ CaCursor ca_seek(const CaArgs &a, const CaLens &L) {
    CaCursor u;
    const long long P = ca_prefix_units(a), K = (long long)a.c.n_kv * a.RT;
    const long long W = P + L.units * K, w = ca_share(a, W);
    const long long n0 = blockIdx.x * w;
    u.stop = min(W, n0 + w);
    u.unit = n0;
    u.prefix = n0 < P;
    u.s = u.h = u.rt = u.t = 0;
    u.T = 1;
    if (n0 >= W) return u;
    long long r;
    if (u.prefix) {
        const int U = ca_units(a.PT), x = (int)ca_div(n0, U);
        u.h = x / a.PRT;
        u.rt = x - u.h * a.PRT;
        u.T = a.PT;
        r = n0 - (long long)x * U;
    } else {
        u.s = L.start;
        u.T = ca_tiles_of(a, L, u.s);
        const int U = ca_units(u.T);
        r = n0 - P - (long long)L.before * K;
        const int y = (int)ca_div(r, U);
        r -= (long long)y * U;
        u.h = y / a.RT;
        u.rt = y - u.h * a.RT;
    }
    if (r < kItemCost) u.unit += kItemCost - r;
    else u.t = (int)r - kItemCost;
    return u;
}
// the next tile (its fields mean nothing once more() is false)
__device__ __forceinline__ void ca_advance(const CaArgs &a, const CaLens &L, CaCursor &u) {
    ++u.unit;
    if (++u.t < u.T) return;
    u.t = 0;
    u.unit += kItemCost;
    if (++u.rt < (u.prefix ? a.PRT : a.RT)) return;
    u.rt = 0;
    if (++u.h < a.c.n_kv) return;
    u.h = 0;
    if (u.prefix) {
        u.prefix = false;
        u.s = 0;
    } else {
        ++u.s;
    }
    for (u.T = 0; u.s < a.c.n_seq && u.T == 0; ++u.s) u.T = ca_tiles_of(a, L, u.s);
    if (u.T > 0) --u.s;                          // the first sequence from there with a tile
    else u.T = 1;
}
__device__ __forceinline__ long long ca_item(const CaArgs &a, const CaCursor &u) {
    return u.prefix ? (long long)u.h * a.PRT + u.rt
                    : (long long)a.c.n_kv * a.PRT + ((long long)u.s * a.c.n_kv + u.h) * a.RT + u.rt;
}

// Row r of an item's tile of query rows: where it lies (null: no such row), and how many
// keys it sees (slots or prefix keys below lim).
__device__ __forceinline__ const __nv_bfloat16 *ca_query(const CaArgs &a, const CaLens &L, const CaCursor &u, int r,
                                                         int *lim = nullptr) {
    int R = u.rt * kCaRows + r, s = u.s;
    if (lim) *lim = 0;
    if (u.prefix) {
        if (R >= a.c.n_seq * a.M) return nullptr;
        s = R / a.M;
        R -= s * a.M;
    } else if (R >= a.M) {
        return nullptr;
    }
    int len, total;
    ca_lens_of(a, L, s, len, total);
    const int i = R / a.G, g = R - i * a.G;
    if (i >= total - len) return nullptr;
    if (lim) *lim = u.prefix ? a.prefix_len : len + i + 1;
    return a.Q + (((size_t)s * a.n_tok + i) * a.n_q + u.h * a.G + g) * a.c.D;
}

}  // namespace crs
