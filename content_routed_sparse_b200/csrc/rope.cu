// Rotary positions and the append of rotated rows to the paged cache, sm_100a.
//
// The rotation moves every element once: it is bound by memory, as long as the angles'
// cost (an fp64 product and reduction, an fp32 sine and cosine) is shared.  A CTA takes a
// few tokens, forms their angles once in shared memory, and walks the tokens' heads in
// memory order, two vectors of pairs in flight per thread and four CTAs per SM.  Walking
// the heads of a token from one thread, with its angles in registers, touched memory in
// 256-byte pieces far apart: 58 us against 47 for 32768 tokens x 16 heads x 128 dims in
// bf16 (268 MB, 5.7 TB/s, 0.89 of the measured copy rate; streaming loads gave the last
// 4 us).  The append of 12 ragged chunks of up to 1000 tokens (32 + 8 + 8 heads, 197 MB
// with the zeroed query rows of absent tokens) takes 41 us with 55% of the issue slots and
// 41% of DRAM used: bound by latency; one token of 64 sequences 3 us.
#include "cache.cuh"

namespace crs {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 2;          // vectors of pairs whose loads are in flight together, per thread
constexpr int kRopePerSm = 4;          // CTAs per SM

template <int BYTES> struct VecOf;
template <> struct VecOf<16> { using type = uint4; };
template <> struct VecOf<8> { using type = uint2; };
template <> struct VecOf<4> { using type = uint32_t; };
template <> struct VecOf<2> { using type = uint16_t; };

// V elements of type T, moved as one access of up to 16 bytes (two for 8 fp32).
template <typename T, int V> struct Pack {
    static constexpr int kBytes = V * (int)sizeof(T) < 16 ? V * (int)sizeof(T) : 16;
    static constexpr int kN = V * (int)sizeof(T) / kBytes;
    using Word = typename VecOf<kBytes>::type;
    union {
        Word w[kN];
        T e[V];
    };
    __device__ Pack() {}
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < kN; ++i) w[i] = __ldcs(reinterpret_cast<const Word *>(p) + i);   // read once
    }
    __device__ __forceinline__ void store(T *p) const {
#pragma unroll
        for (int i = 0; i < kN; ++i) reinterpret_cast<Word *>(p)[i] = w[i];
    }
};

// cos and sin of pos * inv_freq: the angle in turns, reduced in fp64 (its error at
// 2^31 positions is about 2^-22 of a turn), then one fp32 evaluation of the remainder
// in [-1/2, 1/2] turns.
__device__ __forceinline__ void rope_angle(int pos, double inv_freq, float mscale, bool inverse, float &c, float &s) {
    double t = (double)pos * (inv_freq * 0.15915494309189535);    // 1 / (2 pi)
    t -= rint(t);
    sincospif(2.0f * (float)t, &s, &c);
    c *= mscale;
    s *= inverse ? -mscale : mscale;
}

// Where unit u of a head's row lies: units [0, n_rot) are V pairs (vectors at a and b), the
// rest copied: two vectors each where they come in pairs on both sides of the rotated dims,
// else one at a.
template <int V, bool INTER> struct RopeUnit {
    int a, b;
    bool rot, two;
    __device__ __forceinline__ RopeUnit(int u, int n_rot, int rot_begin, int rot_dim, int copied) {
        rot = u < n_rot;
        two = rot || copied > V;
        if (rot) {
            a = rot_begin + u * (INTER ? 2 * V : V);
            b = a + (INTER ? V : rot_dim / 2);
        } else {
            a = (u - n_rot) * copied;
            if (a >= rot_begin) a += rot_dim;
            b = a + V;
        }
    }
};
// elements of a copied unit
inline int rope_copied(const int D, const int rot_begin, const int rot_dim, const int V) {
    return rot_begin % (2 * V) == 0 && (D - rot_begin - rot_dim) % (2 * V) == 0 ? 2 * V : V;
}

// The angles of a CTA's tokens, in shared memory: (cos, sin) of two pairs to 16 bytes (of
// one to 8 when V is 1), the pieces of a unit's V pairs apart, so that the threads of
// neighbouring units read neighbouring 16 bytes.
template <int V> struct RopeTable {
    static constexpr int kPieces = V > 1 ? V / 2 : 1, kPairs = V > 1 ? 2 : 1;
    float *base;
    int tokens, n_rot;
    __device__ __forceinline__ float *at(int t, int u, int piece) const {
        return base + ((piece * tokens + t) * n_rot + u) * (2 * kPairs);
    }
    // pair j of token t
    __device__ __forceinline__ float2 *pair(int t, int j) const {
        const int u = j / V, i = j - u * V;
        return reinterpret_cast<float2 *>(at(t, u, i / kPairs)) + i % kPairs;
    }
    __device__ __forceinline__ void load(int t, int u, float2 (&cs)[V]) const {
        if constexpr (V == 1) {
            cs[0] = *reinterpret_cast<const float2 *>(at(t, u, 0));
        } else {
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                const float4 w = *reinterpret_cast<const float4 *>(at(t, u, p));
                cs[2 * p] = make_float2(w.x, w.y);
                cs[2 * p + 1] = make_float2(w.z, w.w);
            }
        }
    }
};

// (a, b) of V pairs turned in place; interleaved: the pairs are neighbours in a, then b.
template <typename T, int V, bool INTER>
__device__ __forceinline__ void rope_turn(Pack<T, V> &a, Pack<T, V> &b, const float2 (&cs)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        T *pa, *pb;
        if constexpr (INTER && V > 1) {
            Pack<T, V> &w = 2 * i < V ? a : b;               // pair i: elements 2i, 2i + 1 of (a, b)
            pa = &w.e[(2 * i) % V];
            pb = &w.e[(2 * i) % V + 1];
        } else {
            pa = &a.e[i];
            pb = &b.e[i];
        }
        const float x = to_f32(*pa), y = to_f32(*pb);
        *pa = from_f32<T>(x * cs[i].x - y * cs[i].y);
        *pb = from_f32<T>(y * cs[i].x + x * cs[i].y);
    }
}

// n / d for n < 2^31 by one multiplication (d >= 1; the quotient is exact: Granlund and
// Montgomery's round-up method, with the shift and the factor found on the host)
struct FastDiv {
    uint32_t d, mul, shift;
    __device__ __forceinline__ int of(int n) const { return (int)(__umulhi((uint32_t)n, mul) >> shift); }
};
inline FastDiv fast_div(int d) {
    FastDiv f;
    f.d = (uint32_t)d;
    if (d == 1) {                                // n * (2^32 - 1) / 2^32 would be n - 1
        f.mul = 0;
        f.shift = 0;
        return f;
    }
    int l = 0;
    while ((1LL << l) < d) ++l;                  // 2^(l-1) < d <= 2^l
    // m = ceil(2^(31 + l) / d) < 2^32; n m / 2^(31 + l) is exact for n < 2^31
    f.mul = (uint32_t)(((1ULL << (31 + l)) + (uint32_t)d - 1) / (uint32_t)d);
    f.shift = (uint32_t)(l - 1);
    return f;
}
__device__ __forceinline__ int fd_quot(const FastDiv &f, int n) { return f.d == 1 ? n : f.of(n); }

// What a CTA does: it turns `tokens` consecutive tokens, heads [h0, h1) of them.  The
// angles are formed once, in shared memory; the vectors are then walked in memory order
// (unit, head, token), kRopeBatch loads in flight per thread.
constexpr int kRopeMost = 8 * kRopeThreads;      // vectors of pairs of a CTA
constexpr int kRopeSmem = 16384;                 // bytes of (cos, sin) pairs a CTA may hold

template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kRopePerSm)
rope_kernel(const T *x, T *y, const int32_t *__restrict__ pos, const double *__restrict__ inv_freq, int n_tok, int heads,
            int tokens, int per_group, int D, int rot_begin, int rot_dim, long long xs, long long ys, float mscale,
            int inverse, int copied, FastDiv units, FastDiv group) {
    extern __shared__ __align__(16) float rope_cs[];
    const int half = rot_dim / 2, n_rot = half / V;
    const RopeTable<V> table{rope_cs, tokens, n_rot};
    const int t0 = blockIdx.x * tokens, nt = min(tokens, n_tok - t0);
    const int h0 = blockIdx.y * per_group, nh = min(per_group, heads - h0);
    for (int e = threadIdx.x; e < nt * half; e += kRopeThreads) {
        const int t = e / half, j = e - t * half;
        float2 *to = table.pair(t, j);
        rope_angle(pos[t0 + t], inv_freq[j], mscale, inverse != 0, to->x, to->y);
    }
    __syncthreads();
    const int items = nt * per_group * (int)units.d;
    for (int e0 = threadIdx.x; e0 < items; e0 += kRopeThreads * kRopeBatch) {
        Pack<T, V> a[kRopeBatch], b[kRopeBatch];
        T *dst[kRopeBatch];
        int tok[kRopeBatch], unit[kRopeBatch], off[kRopeBatch];      // unit -1: one copied, -2: two; b - a
#pragma unroll
        for (int q = 0; q < kRopeBatch; ++q) {
            const int e = e0 + q * kRopeThreads;
            dst[q] = nullptr;
            if (e >= items) continue;
            const int th = fd_quot(units, e), u = e - th * (int)units.d;
            const int t = fd_quot(group, th), h = th - t * (int)group.d;
            if (h >= nh) continue;
            const RopeUnit<V, INTER> at(u, n_rot, rot_begin, rot_dim, copied);
            const T *row = x + (t0 + t) * xs + (long long)(h0 + h) * D;
            a[q].load(row + at.a);
            if (at.two) b[q].load(row + at.b);
            dst[q] = y + (t0 + t) * ys + (long long)(h0 + h) * D + at.a;
            off[q] = at.b - at.a;
            tok[q] = t;
            unit[q] = at.rot ? u : at.two ? -2 : -1;
        }
#pragma unroll
        for (int q = 0; q < kRopeBatch; ++q) {
            if (!dst[q]) continue;
            if (unit[q] >= 0) {
                float2 cs[V];
                table.load(tok[q], unit[q], cs);
                rope_turn<T, V, INTER>(a[q], b[q], cs);
            }
            if (unit[q] != -1) b[q].store(dst[q] + off[q]);
            a[q].store(dst[q]);
        }
    }
}

// Tokens and head groups of a CTA: up to eight vectors of pairs per thread while that leaves
// some eight CTAs per SM (the angles are shared by the heads of a CTA), less work per CTA
// in smaller calls.
inline void rope_shape(long long n_tok, int heads, int units, int half, int sms, int &tokens, int &groups) {
    const long long vectors = n_tok * heads * units;
    long long per = vectors / ((long long)sms * 8);              // vectors per CTA
    per = per < kRopeThreads ? kRopeThreads : per > kRopeMost ? kRopeMost : per;
    tokens = (int)(per / ((long long)heads * units));
    groups = 1;
    if (tokens < 1) {
        tokens = 1;
        groups = (int)(((long long)heads * units + per - 1) / per);
        if (groups > heads) groups = heads;
    }
    const int most = half > 0 ? kRopeSmem / (half * 8) : tokens;
    if (tokens > most && most >= 1) tokens = most;
    if (tokens > n_tok) tokens = (int)n_tok;
}

template <typename T, int V>
int rope_launch(const crs_rope_params *p, int n_tok, int heads, const void *x, long long xs, const int32_t *pos,
                const double *inv_freq, void *y, long long ys, cudaStream_t s) {
    const int half = p->rot_dim / 2, copied = rope_copied(p->D, p->rot_begin, p->rot_dim, V);
    const int units = half / V + (p->D - p->rot_dim) / copied;
    int tokens, groups;
    rope_shape(n_tok, heads, units, half, cache_sms(), tokens, groups);
    const int per_group = ceil_div(heads, groups);
    const dim3 grid((unsigned)ceil_div(n_tok, tokens), (unsigned)ceil_div(heads, per_group));
    const size_t smem = (size_t)tokens * half * 8;
    const FastDiv du = fast_div(units), dg = fast_div(per_group);
    ProfScope _ps(K_ROPE, s);
    auto kern = p->interleaved ? rope_kernel<T, V, true> : rope_kernel<T, V, false>;
    kern<<<grid, kRopeThreads, smem, s>>>(static_cast<const T *>(x), static_cast<T *>(y), pos, inv_freq, n_tok, heads,
                                          tokens, per_group, p->D, p->rot_begin, p->rot_dim, xs, ys, p->mscale,
                                          p->inverse, copied, du, dg);
    return cudaGetLastError() == cudaSuccess ? CRS_OK : CRS_ERR_CUDA;
}

inline int rope_validate(const crs_rope_params *p) {
    if (!p) return CRS_ERR_INVALID_ARG;
    if (p->D < 1 || p->rot_begin < 0 || p->rot_dim < 0 || (p->rot_dim & 1)) return CRS_ERR_INVALID_ARG;
    if ((long long)p->rot_begin + p->rot_dim > p->D) return CRS_ERR_INVALID_ARG;
    if (p->D > 1024) return CRS_ERR_UNSUPPORTED;
    return CRS_OK;
}

// ------------------------------------------------------------------- cache append --
struct AppendArgs {
    CacheDev c;
    const __nv_bfloat16 *k, *v, *q;
    __nv_bfloat16 *q_out;
    long long ks, vs, qs;
    const double *inv_freq;
    const int32_t *n_new;
    int n_tok, n_q, rot_begin, rot_dim, tokens, per_group, inverse, copied;
    float mscale;
    FastDiv units, group;
};
constexpr int kApTokens = 64;                    // tokens of a CTA at most

// As rope_kernel, over the heads k, v, q of the batch's tokens; where a token's rows go is
// found once per token.
template <bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kRopePerSm) cache_append_kernel(AppendArgs a) {
    constexpr int V = 8;
    using P = Pack<__nv_bfloat16, V>;
    extern __shared__ __align__(16) float rope_cs[];
    __shared__ int rows[kApTokens];              // row in the pools; -1: no row; -2: not a token
    const int half = a.rot_dim / 2, n_rot = half / V, n_kv = a.c.n_kv, D = a.c.D;
    const RopeTable<V> table{rope_cs, a.tokens, n_rot};
    const int all = a.c.n_seq * a.n_tok;
    const int t0 = blockIdx.x * a.tokens, nt = min(a.tokens, all - t0);
    const int h0 = blockIdx.y * a.per_group, nh = min(a.per_group, 2 * n_kv + a.n_q - h0);
    if (threadIdx.x < nt) {
        const int tok = t0 + threadIdx.x, s = tok / a.n_tok, i = tok - s * a.n_tok;
        const int len = cache_len(a.c, s), n = cache_new(a.c, a.n_new, a.n_tok, s, len);
        const int asked = a.n_new ? min(max(a.n_new[s], 0), a.n_tok) : a.n_tok;
        if (i >= n && i < asked && h0 == 0) raise_error(CRS_DEVERR_CAPACITY);
        const bool stores = h0 < 2 * n_kv;
        rows[threadIdx.x] = i >= n ? -2 : stores ? cache_row(a.c, s, len + i) : -1;
        if (i < n) {
            const int position = a.c.next_pos[s] + i;
            for (int h = h0; h < min(n_kv, h0 + nh); ++h) {
                const size_t m = ((size_t)s * n_kv + h) * a.c.cap + len + i;
                if (a.c.pos) a.c.pos[m] = position;
                if (a.c.mass) a.c.mass[m] = 0.0f;
            }
        }
    }
    for (int e = threadIdx.x; e < nt * half; e += kRopeThreads) {
        const int t = e / half, j = e - t * half, tok = t0 + t, s = tok / a.n_tok;
        float2 *to = table.pair(t, j);
        rope_angle(a.c.next_pos[s] + (tok - s * a.n_tok), a.inv_freq[j], a.mscale, a.inverse != 0, to->x, to->y);
    }
    __syncthreads();
    const int items = nt * a.per_group * (int)a.units.d;
    for (int e0 = threadIdx.x; e0 < items; e0 += kRopeThreads * kRopeBatch) {
        P x[kRopeBatch], y[kRopeBatch];
        __nv_bfloat16 *dst[kRopeBatch];
        int at_t[kRopeBatch], unit[kRopeBatch], off[kRopeBatch];     // unit -1: one vector, -2: two as they are; b - a
#pragma unroll
        for (int q = 0; q < kRopeBatch; ++q) {
            const int e = e0 + q * kRopeThreads;
            dst[q] = nullptr;
            if (e >= items) continue;
            const int th = fd_quot(a.units, e), u = e - th * (int)a.units.d;
            const int t = fd_quot(a.group, th), hg = th - t * (int)a.group.d, h = h0 + hg;
            if (hg >= nh) continue;
            const int row = rows[t];
            const long long tok = t0 + t;
            const RopeUnit<V, INTER> at(u, n_rot, a.rot_begin, a.rot_dim, a.copied);
            const __nv_bfloat16 *src;
            bool turn = true;
            if (h < 2 * n_kv) {
                if (row < 0) continue;
                turn = h < n_kv;
                const int kh = turn ? h : h - n_kv;
                src = (turn ? a.k + tok * a.ks : a.v + tok * a.vs) + (size_t)kh * D;
                dst[q] = (turn ? a.c.k : a.c.v) + ((size_t)row * n_kv + kh) * D;
            } else {
                src = a.q + tok * a.qs + (size_t)(h - 2 * n_kv) * D;
                dst[q] = a.q_out + ((size_t)tok * a.n_q + (h - 2 * n_kv)) * D;
            }
            if (row != -2) {
                x[q].load(src + at.a);
                if (at.two) y[q].load(src + at.b);
            } else {                             // the query row of a token that is not one: zeros
                x[q].w[0] = y[q].w[0] = make_uint4(0u, 0u, 0u, 0u);
                turn = false;
            }
            dst[q] += at.a;
            off[q] = at.b - at.a;
            at_t[q] = t;
            unit[q] = !at.two ? -1 : at.rot && turn ? u : -2;
        }
#pragma unroll
        for (int q = 0; q < kRopeBatch; ++q) {
            if (!dst[q]) continue;
            if (unit[q] >= 0) {
                float2 cs[V];
                table.load(at_t[q], unit[q], cs);
                rope_turn<__nv_bfloat16, V, INTER>(x[q], y[q], cs);
            }
            if (unit[q] != -1) y[q].store(dst[q] + off[q]);
            x[q].store(dst[q]);
        }
    }
}

__global__ void cache_commit_kernel(CacheDev c, int n_tok, const int32_t *accepted) {
    const int s = blockIdx.x * blockDim.x + threadIdx.x;
    if (s >= c.n_seq) return;
    const int len = cache_len(c, s), n = cache_new(c, accepted, n_tok, s, len);
    c.seq_len[s] = len + n;
    c.next_pos[s] += n;
}

}  // namespace crs

using namespace crs;

extern "C" int crs_rope(const crs_rope_params *p, int n_tok, int n_heads, int dtype, const void *x, int64_t x_stride,
                        const int32_t *pos, const double *inv_freq, void *y, int64_t y_stride, void *stream) {
    int st = rope_validate(p);
    if (st) return st;
    if (n_tok < 0 || n_heads < 1 || (dtype != CRS_F32 && dtype != CRS_BF16)) return CRS_ERR_INVALID_ARG;
    if (n_heads > 65535) return CRS_ERR_UNSUPPORTED;
    if (n_tok == 0) return CRS_OK;
    if (!x || !y || !pos || (p->rot_dim > 0 && !inv_freq)) return CRS_ERR_INVALID_ARG;
    if (x_stride < (int64_t)n_heads * p->D || y_stride < (int64_t)n_heads * p->D) return CRS_ERR_INVALID_ARG;
    if (x == y && x_stride != y_stride) return CRS_ERR_INVALID_ARG;
    const int size = dtype == CRS_F32 ? 4 : 2;
    // one bit set per power of two that some offset, stride or address lacks
    const uint64_t odd = (uint64_t)(p->interleaved ? p->rot_dim : p->rot_dim / 2) | (uint64_t)p->rot_begin |
                         (uint64_t)p->D | (uint64_t)x_stride | (uint64_t)y_stride |
                         (uint64_t)(reinterpret_cast<uintptr_t>(x) / size) |
                         (uint64_t)(reinterpret_cast<uintptr_t>(y) / size) |
                         (p->interleaved ? (uint64_t)(p->rot_dim / 2) : 0);
    if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) & (uintptr_t)(size - 1))
        return CRS_ERR_INVALID_ARG;
    const int v = (odd & 1) ? 1 : (odd & 2) ? 2 : (odd & 4) ? 4 : 8;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
#define CRS_ROPE_CASE(T, V) \
    return rope_launch<T, V>(p, n_tok, n_heads, x, x_stride, pos, inv_freq, y, y_stride, s)
    if (dtype == CRS_F32) {
        if (v == 8) CRS_ROPE_CASE(float, 8);
        if (v == 4) CRS_ROPE_CASE(float, 4);
        if (v == 2) CRS_ROPE_CASE(float, 2);
        CRS_ROPE_CASE(float, 1);
    }
    if (v == 8) CRS_ROPE_CASE(__nv_bfloat16, 8);
    if (v == 4) CRS_ROPE_CASE(__nv_bfloat16, 4);
    if (v == 2) CRS_ROPE_CASE(__nv_bfloat16, 2);
    CRS_ROPE_CASE(__nv_bfloat16, 1);
#undef CRS_ROPE_CASE
}

extern "C" int crs_cache_append(const crs_cache_params *p, const crs_cache_state *st, const crs_rope_params *r,
                                const double *inv_freq, int n_tok, const int32_t *n_new, const void *k,
                                int64_t k_stride, const void *v, int64_t v_stride, const void *q, int64_t q_stride,
                                int n_q, void *q_out, void *stream) {
    int e = cache_validate(p);
    if (e) return e;
    if (r) {
        if ((e = rope_validate(r))) return e;
        if (r->D != p->D) return CRS_ERR_INVALID_ARG;
        if (r->rot_begin % 8 || r->rot_dim % 16) return CRS_ERR_UNSUPPORTED;
    }
    if (n_tok < 1 || n_q < 0) return CRS_ERR_INVALID_ARG;
    if ((e = cache_check_state(st))) return e;
    if (!k || !v || (r && r->rot_dim > 0 && !inv_freq)) return CRS_ERR_INVALID_ARG;
    const bool with_q = q != nullptr;
    if (with_q && (!q_out || n_q < 1 || q_stride < (int64_t)n_q * p->D)) return CRS_ERR_INVALID_ARG;
    if (k_stride < (int64_t)p->n_kv * p->D || v_stride < (int64_t)p->n_kv * p->D) return CRS_ERR_INVALID_ARG;
    if ((k_stride | v_stride | (with_q ? q_stride : 0)) & 7) return CRS_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(q) |
         (with_q ? reinterpret_cast<uintptr_t>(q_out) : 0)) & 15)
        return CRS_ERR_INVALID_ARG;
    AppendArgs a;
    a.c = cache_dev(p, st);
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.q_out = static_cast<__nv_bfloat16 *>(q_out);
    a.ks = k_stride;
    a.vs = v_stride;
    a.qs = q_stride;
    a.inv_freq = inv_freq;
    a.n_new = n_new;
    a.n_tok = n_tok;
    a.n_q = with_q ? n_q : 0;
    a.rot_begin = r ? r->rot_begin : 0;
    a.rot_dim = r ? r->rot_dim : 0;
    a.inverse = r ? r->inverse : 0;
    a.mscale = r ? r->mscale : 1.0f;
    a.copied = rope_copied(p->D, a.rot_begin, a.rot_dim, 8);
    const int heads = 2 * p->n_kv + a.n_q, units = a.rot_dim / 16 + (p->D - a.rot_dim) / a.copied;
    const long long toks = (long long)p->n_seq * n_tok;
    if (toks > 0x7fffffffLL || heads > 65535) return CRS_ERR_UNSUPPORTED;
    int groups;
    rope_shape(toks, heads, units, a.rot_dim / 2, cache_sms(), a.tokens, groups);
    a.tokens = min(a.tokens, kApTokens);
    a.per_group = ceil_div(heads, groups);
    a.units = fast_div(units);
    a.group = fast_div(a.per_group);
    const dim3 grid((unsigned)ceil_div_ll(toks, a.tokens), (unsigned)ceil_div(heads, a.per_group));
    const size_t smem = (size_t)a.tokens * a.rot_dim * 4;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    {
        ProfScope _ps(K_CACHE_APPEND, s);
        if (r && r->interleaved) cache_append_kernel<true><<<grid, kRopeThreads, smem, s>>>(a);
        else cache_append_kernel<false><<<grid, kRopeThreads, smem, s>>>(a);
    }
    CRS_CHECK_LAUNCH();
    return CRS_OK;
}

extern "C" int crs_cache_commit(const crs_cache_params *p, const crs_cache_state *st, int n_tok,
                                const int32_t *accepted, void *stream) {
    int e = cache_validate(p);
    if (e) return e;
    if (n_tok < 0) return CRS_ERR_INVALID_ARG;
    if ((e = cache_check_state(st))) return e;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    {
        ProfScope _ps(K_CACHE_APPEND, s);
        cache_commit_kernel<<<ceil_div(p->n_seq, 256), 256, 0, s>>>(cache_dev(p, st), n_tok, accepted);
    }
    CRS_CHECK_LAUNCH();
    return CRS_OK;
}
