// Selection of the slots to keep by accumulated attention weight, and the eviction of
// the others from the paged cache, sm_100a.
//
// Selection: one CTA per (sequence, KV head) holds the slots' order-preserving 32-bit
// keys in registers, consecutive slots per warp.  The keep-th largest key is bracketed by
// a sample and found among the few keys in the bracket, by counts alone (no order of
// arrival enters the result); a scan of the warps' counts above and at it, and ballots,
// place the kept slots in ascending order, ties to the lower slot.  Caches longer than the
// registers hold re-read the keys from memory: four passes with 256-bin histograms, then
// the same placement.
//
// Bound by issue (62%) and the barriers between the passes: 32 sequences x 4 heads of 30000
// to 32768 slots to 4096 take 23 to 29 us; 8 of them are the 34 MB of weights and positions,
// the rest passes over 32 keys per thread, of which every instruction costs about 0.15 us:
// one pass counts the bracket, one gathers it, two place.
//
// Eviction: nothing depends on the order of a head's slots, so only the kept slots
// past the new length move, each into a free slot below it: the r-th of the former
// into the r-th of the latter (354 MB read and written in 256-byte rows at random: 74 us,
// 4.8 TB/s).  Both are found by binary search in the ascending list
// (the free slots before entry i number idx[i] - i), so every warp finds its own
// moves; sources and destinations are disjoint, and the moves run in any order.
#include "cache.cuh"

namespace crs {

struct MassSelArgs {
    const float *mass;
    const int32_t *pos, *seq_len, *next_pos;
    int32_t *idx, *count;
    int n_kv, cap, keep, sink_end, window;
};

__device__ __forceinline__ uint32_t sel_key(float m, int pos, bool has_pos, int sink_end, int recent, bool &nan) {
    if (has_pos && (pos < sink_end || pos >= recent)) return 0xffffffffu;
    nan |= m != m;
    return score_key(m);
}

// exclusive scan over the CTA of one value per thread (blockDim.x a multiple of 32, one barrier)
__device__ __forceinline__ uint32_t cta_scan(uint32_t v, uint32_t *warp_sums, uint32_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
    uint32_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    uint32_t w = lane < n_warps ? warp_sums[lane] : 0u;
    uint32_t winc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, winc, o);
        if (lane >= o) winc += u;
    }
    total = __shfl_sync(0xffffffffu, winc, 31);
    return inc - v + __shfl_sync(0xffffffffu, winc - w, warp);
}

// Warp w holds the 32 KPT slots from w 32 KPT, slot i 32 + lane of them in lane's key[i]:
// loads and the kept slots' stores are contiguous, and ballots rank the slots in order.
template <int THREADS, int KPT>
__global__ void __launch_bounds__(THREADS) mass_select_kernel(MassSelArgs a) {
    // keys between at most, sample size, bins of the sample's histogram (in the list's place)
    constexpr int kList = THREADS >= 1024 ? 6 * THREADS : 1024, kSample = THREADS >= 1024 ? 512 : 256;
    constexpr int kBins = THREADS >= 1024 ? 4096 : 1024, kDigit = THREADS >= 1024 ? 20 : 22;
    __shared__ uint32_t sums[32], pick[2], list[kList];
    const int sh = blockIdx.x, s = sh / a.n_kv, h = sh - s * a.n_kv;
    const int tid = threadIdx.x, lane = tid & 31;
    const int len = min(max(a.seq_len[s], 0), a.cap), k = min(a.keep, len);
    int32_t *out = a.idx + (size_t)sh * a.keep;
    if (h == 0 && tid == 0) a.count[s] = k;
    for (int i = k + tid; i < a.keep; i += THREADS) out[i] = -1;
    if (len <= a.keep) {
        for (int i = tid; i < len; i += THREADS) out[i] = i;
        return;
    }
    const float *mass = a.mass + (size_t)sh * a.cap;
    const int32_t *pos = a.pos ? a.pos + (size_t)sh * a.cap : nullptr;
    const int recent = a.pos ? a.next_pos[s] - a.window : 0;
    const int j0 = (tid >> 5) * (32 * KPT) + lane;
    uint32_t key[KPT];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
        const int j = j0 + i * 32;
        key[i] = j < len ? __float_as_uint(mass[j]) : 0u;
    }
    // 16 positions at a time: all 2 KPT loads in flight would need the registers twice
#pragma unroll
    for (int i0 = 0; i0 < KPT; i0 += 16) {
        int p[KPT < 16 ? KPT : 16];
#pragma unroll
        for (int i = 0; i < (KPT < 16 ? KPT : 16); ++i) {
            const int j = j0 + (i0 + i) * 32;
            p[i] = pos && j < len ? pos[j] : 0;
        }
#pragma unroll
        for (int i = 0; i < (KPT < 16 ? KPT : 16); ++i) {
            const int j = j0 + (i0 + i) * 32;
            key[i0 + i] = j < len ? sel_key(__uint_as_float(key[i0 + i]), p[i], pos != nullptr, a.sink_end, recent, nan) : 0u;
        }
    }
    if (nan) raise_error(CRS_DEVERR_NONFINITE);
    // T, the k-th largest key: c(lo) >= k > c(hi) is kept for c(x), the number of keys that
    // reach x.  A sample (the first slot of some threads) gives a narrow pair lo, hi by a
    // histogram of its top digits; the few keys between go to shared memory, and byte by byte
    // histograms of them find T.  Where the sample misleads, or too many keys lie between,
    // bisection over all keys goes on.
    for (int e = tid; e < kBins; e += THREADS) list[e] = 0u;
    __syncthreads();
    if (tid % (THREADS / kSample) == 0) atomicAdd(&list[key[0] >> kDigit], 1u);
    __syncthreads();
    {
        // the sample's ranks 3.5 deviations before and after k's (absent slots are sampled too)
        const float share = (float)k / (float)(THREADS * KPT);
        const float mid = share * kSample, dev = 3.5f * sqrtf(mid * (1.0f - share)) + 2.0f;
        const uint32_t up = (uint32_t)max(0, (int)(mid - dev)), down = (uint32_t)(mid + dev) + 1u;
        if (tid == 0) {
            pick[0] = 0u;
            pick[1] = 0xffffffffu;               // reached by protected slots only
        }
        constexpr int per = kBins / THREADS;
        const int top = kBins - 1 - tid * per;   // this thread's bins, from the top
        uint32_t sum = 0, total;
#pragma unroll
        for (int e = 0; e < per; ++e) sum += list[top - e];
        uint32_t above = cta_scan(sum, sums, total);
        if ((above < up && up <= above + sum) || (above < down && down <= above + sum)) {
            for (int e = 0; e < per; ++e) {
                const uint32_t c = list[top - e];
                const uint32_t from = (uint32_t)(top - e) << kDigit;
                if (above < up && up <= above + c && top - e < kBins - 1) pick[1] = from + (1u << kDigit);
                if (above < down && down <= above + c) pick[0] = from;
                above += c;
            }
        }
        __syncthreads();
    }
    uint32_t lo = pick[0], hi = pick[1];
    int ph = 0;
    auto reach = [&](uint32_t x) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < KPT; ++i) n += key[i] >= x;
        return cta_count(n, ph);
    };
    int n_lo, n_hi;
    {
        uint32_t n = 0;                          // both counts at once: at most 2^15 keys
#pragma unroll
        for (int i = 0; i < KPT; ++i) n += (key[i] >= lo ? 1u : 0u) + (key[i] >= hi ? 0x10000u : 0u);
        n = (uint32_t)cta_count((int)n, ph);
        n_lo = (int)(n & 0xffffu);
        n_hi = (int)(n >> 16);
    }
    if (n_hi >= k) {                             // enough keys reach hi: T is hi or above
        lo = hi;
        n_lo = n_hi;
        hi = 0xffffffffu;
        n_hi = lo == hi ? 0 : reach(hi);
        if (n_hi >= k) lo = hi;                  // protected slots alone
    } else if (n_lo < k) {
        hi = lo;
        n_hi = n_lo;
        lo = 0u;
        n_lo = THREADS * KPT;
    }
    if (hi - lo > 1u && n_lo - n_hi <= kList) {
        uint32_t mine = 0, total;
#pragma unroll
        for (int i = 0; i < KPT; ++i) mine += key[i] - lo < hi - lo;
        uint32_t at = cta_scan(mine, sums, total);
#pragma unroll
        for (int i = 0; i < KPT; ++i)
            if (key[i] - lo < hi - lo) list[at++] = key[i] - lo;
        __syncthreads();
        constexpr int kFew = kList / THREADS;
        const int n = n_lo - n_hi;
        uint32_t few[kFew], left = (uint32_t)(k - n_hi), d = 0u;     // d: T - lo, its bytes so far
#pragma unroll
        for (int i = 0; i < kFew; ++i) few[i] = i * THREADS + tid < n ? list[i * THREADS + tid] : 0u;
        __syncthreads();
        for (int shift = max(0, 24 - __clz(hi - lo - 1u)), up = 32;; up = shift, shift = max(0, shift - 8)) {
            // the digit [shift, up) of the keys that share the bits from `up` on
            if (tid < 256) list[tid] = 0u;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kFew; ++i)
                if (i * THREADS + tid < n && (up == 32 || (few[i] ^ d) >> up == 0u))
                    atomicAdd(&list[(few[i] >> shift) & ((1u << min(8, up - shift)) - 1u)], 1u);
            __syncthreads();
            const uint32_t own = tid < 256 ? list[255 - tid] : 0u;
            const uint32_t above = cta_scan(own, sums, total);
            if (above < left && left <= above + own) {
                pick[0] = 255u - tid;
                pick[1] = left - above;
            }
            __syncthreads();
            d |= pick[0] << shift;
            left = pick[1];
            if (shift == 0) break;
        }
        lo += d;
        hi = lo + 1u;
    }
    while (hi - lo > 1u) {
        const uint32_t x = lo + ((hi - lo) >> 1);
        if (reach(x) >= k) lo = x;
        else hi = x;
    }
    const uint32_t T = lo;
    // Slots past len have key 0 and follow every slot of the sequence: they lose every tie (a
    // tie at key 0 that is kept whole, `ties` false, cannot include them: they count in it)
    uint32_t gt = 0, eq = 0;
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
        gt += key[i] > T;
        eq += key[i] == T;
    }
    // the warp's slots above the threshold and at it, and those of the warps before it
    const uint32_t own = __reduce_add_sync(0xffffffffu, gt | (eq << 16));
    uint32_t total;
    const uint32_t before = __shfl_sync(0xffffffffu, cta_scan(lane == 0 ? own : 0u, sums, total), 0);
    const uint32_t need = (uint32_t)k - (total & 0xffffu);
    const bool ties = (total >> 16) != need;     // else every key equal to T is kept
    uint32_t eb = before >> 16, at = (before & 0xffffu) + min(eb, need);
    const uint32_t lower = (1u << lane) - 1u;
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
        bool take = key[i] >= T;
        if (ties) {
            const uint32_t e = __ballot_sync(0xffffffffu, key[i] == T);
            take = key[i] > T || (key[i] == T && eb + __popc(e & lower) < need);
            eb += __popc(e);
        }
        const uint32_t t = __ballot_sync(0xffffffffu, take);
        if (take) out[at + __popc(t & lower)] = j0 + i * 32;
        at += __popc(t);
    }
}

// Any length: the keys stay in memory.
constexpr int kMassThreads = 1024;
__global__ void __launch_bounds__(kMassThreads) mass_select_long_kernel(MassSelArgs a) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t sums[32];
    __shared__ uint32_t pick[2];
    const int sh = blockIdx.x, s = sh / a.n_kv, h = sh - s * a.n_kv;
    const int tid = threadIdx.x;
    const int len = min(max(a.seq_len[s], 0), a.cap), k = min(a.keep, len);
    int32_t *out = a.idx + (size_t)sh * a.keep;
    if (h == 0 && tid == 0) a.count[s] = k;
    for (int i = k + tid; i < a.keep; i += kMassThreads) out[i] = -1;
    if (len <= a.keep) {
        for (int i = tid; i < len; i += kMassThreads) out[i] = i;
        return;
    }
    const float *mass = a.mass + (size_t)sh * a.cap;
    const int32_t *pos = a.pos ? a.pos + (size_t)sh * a.cap : nullptr;
    const int recent = a.pos ? a.next_pos[s] - a.window : 0;
    bool nan = false;
    auto key_of = [&](int j) {
        return sel_key(mass[j], pos ? pos[j] : 0, pos != nullptr, a.sink_end, recent, nan);
    };
    // byte by byte from the top: the bin that holds the k-th largest key
    uint32_t T = 0u, left = (uint32_t)k;
    for (int b = 24; b >= 0; b -= 8) {
        if (tid < 256) hist[tid] = 0u;
        __syncthreads();
        for (int j = tid; j < len; j += kMassThreads) {
            const uint32_t key = key_of(j);
            if (b == 24 || (key >> (b + 8)) == (T >> (b + 8))) {
                // the keys of a warp mostly share a bin: one addition per group of equal bins
                const uint32_t bin = (key >> b) & 255u;
                const unsigned grp = __match_any_sync(__activemask(), bin);
                if ((int)(tid & 31) == __ffs(grp) - 1) atomicAdd(&hist[bin], (uint32_t)__popc(grp));
            }
        }
        __syncthreads();
        const uint32_t own = tid < 256 ? hist[255 - tid] : 0u;       // bins from the top
        uint32_t total;
        const uint32_t above = cta_scan(own, sums, total);
        if (tid < 256 && above < left && left <= above + own) {
            pick[0] = 255u - tid;
            pick[1] = left - above;
        }
        __syncthreads();
        T |= pick[0] << b;
        left = pick[1];
        __syncthreads();
    }
    if (nan) raise_error(CRS_DEVERR_NONFINITE);
    // left = how many of the keys equal to T are kept; slots in order, 1024 at a time
    uint32_t kept = 0, ties = 0;
    for (int j0 = 0; j0 < len; j0 += kMassThreads) {
        const int j = j0 + tid;
        const uint32_t key = j < len ? key_of(j) : 0u;
        const uint32_t gt = j < len && key > T, eq = j < len && key == T;
        uint32_t total;
        const uint32_t before = cta_scan(gt | (eq << 16), sums, total);
        const uint32_t eb = ties + (before >> 16);
        const uint32_t at = kept + (before & 0xffffu) + min(eb, left);
        if (gt || (eq && eb < left)) out[at] = j;
        kept += total & 0xffffu;
        ties += total >> 16;
        __syncthreads();                         // sums is reused
    }
}

// --------------------------------------------------------------------------- evict --
constexpr int kEvWarps = 4;
constexpr int kEvBatch = 8;                      // row copies a warp keeps in flight

template <int D>
__global__ void __launch_bounds__(kEvWarps * 32)
cache_evict_kernel(CacheDev c, int keep, const int32_t *__restrict__ idx, const int32_t *__restrict__ count,
                   int blocks) {                 // CTAs per (sequence, KV head)
    constexpr int kLanes = D / 4;                // lanes per move: D / 8 for K, D / 8 for V
    constexpr int kPer = 32 / kLanes;            // moves per warp access
    const int sh = blockIdx.x / blocks, block = blockIdx.x - sh * blocks;
    const int s = sh / c.n_kv, h = sh - s * c.n_kv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = min(max(count[s], 0), min(keep, c.cap));
    if (block == 0 && h == 0 && threadIdx.x == 0) c.seq_len[s] = n;
    const int32_t *list = idx + (size_t)sh * keep;
    int lo = 0, hi = n;                          // entries below n
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (list[mid] < n) lo = mid + 1;
        else hi = mid;
    }
    const int stay = lo, moves = n - stay;
    const int r = (block * kEvWarps + warp) * 32 + lane;
    if (r - lane >= moves) return;               // whole warps
    int src = -1, dst = -1;
    if (r < moves) {
        const int from = list[stay + r];
        int b = 0, e = stay;                     // the first kept slot with more than r free ones before it
        while (b < e) {
            const int mid = (b + e) >> 1;
            if (list[mid] - mid > r) e = mid;
            else b = mid + 1;
        }
        const int to = r + b;
        if (from >= 0 && from < c.cap) {
            src = cache_row(c, s, from);
            dst = cache_row(c, s, to);
            if (src >= 0 && dst >= 0) {
                const size_t base = (size_t)sh * c.cap;
                if (c.pos) c.pos[base + to] = c.pos[base + from];
                if (c.mass) c.mass[base + to] = c.mass[base + from];
            }
        } else {
            raise_error(CRS_DEVERR_INDEX);
        }
    }
    const int which = lane / kLanes, part = lane % kLanes;
    __nv_bfloat16 *pool = (part < D / 8 ? c.k : c.v) + (size_t)h * D + (part % (D / 8)) * 8;
    const size_t stride = (size_t)c.n_kv * D;
#pragma unroll
    for (int b = 0; b < 32; b += kEvBatch * kPer) {
        uint4 v[kEvBatch];
        int to[kEvBatch];
#pragma unroll
        for (int q = 0; q < kEvBatch; ++q) {
            const int m = b + q * kPer + which;
            const int from = __shfl_sync(0xffffffffu, src, m);
            to[q] = __shfl_sync(0xffffffffu, dst, m);
            if (from < 0) to[q] = -1;
            if (to[q] >= 0) v[q] = *reinterpret_cast<const uint4 *>(pool + (size_t)from * stride);
        }
#pragma unroll
        for (int q = 0; q < kEvBatch; ++q)
            if (to[q] >= 0) *reinterpret_cast<uint4 *>(pool + (size_t)to[q] * stride) = v[q];
    }
}

}  // namespace crs

using namespace crs;

extern "C" int crs_mass_select(const crs_mass_select_params *p, const float *mass, const int32_t *pos,
                               const int32_t *seq_len, const int32_t *next_pos, int32_t *idx, int32_t *count,
                               void *stream) {
    if (!p || p->n_seq < 1 || p->n_kv < 1 || p->cap < 1 || p->keep < 1 || p->keep > p->cap || p->window < 0)
        return CRS_ERR_INVALID_ARG;
    const long long ctas = (long long)p->n_seq * p->n_kv;
    if (ctas > 0x7fffffffLL) return CRS_ERR_UNSUPPORTED;
    if (!mass || !seq_len || !idx || !count || (pos && !next_pos)) return CRS_ERR_INVALID_ARG;
    // a sequence's heads run side by side: what one writes, the others must not read
    const void *in[4] = {mass, pos, seq_len, pos ? next_pos : nullptr};
    for (const void *q : in)
        if (q && (q == idx || q == count)) return CRS_ERR_INVALID_ARG;
    if (idx == count) return CRS_ERR_INVALID_ARG;
    MassSelArgs a{mass, pos, seq_len, next_pos, idx, count, p->n_kv, p->cap, p->keep, p->sink_end, p->window};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)ctas;
    {
        ProfScope _ps(K_MASS_SELECT, s);
        if (p->cap <= 1024) mass_select_kernel<256, 4><<<grid, 256, 0, s>>>(a);
        else if (p->cap <= 2048) mass_select_kernel<256, 8><<<grid, 256, 0, s>>>(a);
        else if (p->cap <= 4096) mass_select_kernel<512, 8><<<grid, 512, 0, s>>>(a);
        else if (p->cap <= 8192) mass_select_kernel<1024, 8><<<grid, 1024, 0, s>>>(a);
        else if (p->cap <= 16384) mass_select_kernel<1024, 16><<<grid, 1024, 0, s>>>(a);
        else if (p->cap <= 32768) mass_select_kernel<1024, 32><<<grid, 1024, 0, s>>>(a);
        else mass_select_long_kernel<<<grid, kMassThreads, 0, s>>>(a);
    }
    CRS_CHECK_LAUNCH();
    return CRS_OK;
}

extern "C" int crs_cache_evict(const crs_cache_params *p, const crs_cache_state *st, int keep, const int32_t *idx,
                               const int32_t *count, void *stream) {
    int e = cache_validate(p);
    if (e) return e;
    if (keep < 1) return CRS_ERR_INVALID_ARG;
    if ((e = cache_check_state(st))) return e;
    if (!idx || !count) return CRS_ERR_INVALID_ARG;
    const long long sh = (long long)p->n_seq * p->n_kv;
    // n kept slots of cap: at most min(n, cap - n) move
    const int most = max(1, min(keep, p->cap / 2));
    const int blocks = ceil_div(most, kEvWarps * 32);
    if (sh * blocks > 0x7fffffffLL) return CRS_ERR_UNSUPPORTED;
    const unsigned grid = (unsigned)(sh * blocks);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const CacheDev c = cache_dev(p, st);
    {
        ProfScope _ps(K_CACHE_EVICT, s);
        if (p->D == 128) cache_evict_kernel<128><<<grid, kEvWarps * 32, 0, s>>>(c, keep, idx, count, blocks);
        else cache_evict_kernel<64><<<grid, kEvWarps * 32, 0, s>>>(c, keep, idx, count, blocks);
    }
    CRS_CHECK_LAUNCH();
    return CRS_OK;
}
