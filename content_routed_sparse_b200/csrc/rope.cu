// Rotary positions and the append of rotated rows to the paged cache, sm_100a.
//
// The rotation moves every element once: it is bound by memory.  A thread owns one
// vector of pairs of one token, forms their cosines and sines once, and applies them
// to several heads (they do not depend on the head), so the angle's cost is shared;
// with few tokens the heads are spread over threads instead.
#include "cache.cuh"

namespace crs {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;          // heads whose loads are in flight together

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
        for (int i = 0; i < kN; ++i) w[i] = reinterpret_cast<const Word *>(p)[i];
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

// Where unit u of a head's row lies: units [0, n_rot) are V pairs (vectors at a and
// b), the rest V copied elements at a.
template <int V, bool INTER> struct RopeUnit {
    int a, b;
    bool rot;
    __device__ __forceinline__ RopeUnit(int u, int n_rot, int rot_begin, int rot_dim) {
        rot = u < n_rot;
        if (rot) {
            a = rot_begin + u * (INTER ? 2 * V : V);
            b = a + (INTER ? V : rot_dim / 2);
        } else {
            a = (u - n_rot) * V;
            if (a >= rot_begin) a += rot_dim;
            b = a;
        }
    }
};

// (a, b) of V pairs turned in place; interleaved: the pairs are neighbours in a, then b.
template <typename T, int V, bool INTER>
__device__ __forceinline__ void rope_turn(Pack<T, V> &a, Pack<T, V> &b, const float (&c)[V], const float (&s)[V]) {
    if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            Pack<T, V> &w = 2 * i < V ? a : b;               // pair i: elements 2i, 2i + 1 of (a, b)
            const int at = (2 * i) % V;
            if constexpr (V == 1) {
                const float x = to_f32(a.e[0]), y = to_f32(b.e[0]);
                a.e[0] = from_f32<T>(x * c[0] - y * s[0]);
                b.e[0] = from_f32<T>(y * c[0] + x * s[0]);
            } else {
                const float x = to_f32(w.e[at]), y = to_f32(w.e[at + 1]);
                w.e[at] = from_f32<T>(x * c[i] - y * s[i]);
                w.e[at + 1] = from_f32<T>(y * c[i] + x * s[i]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float x = to_f32(a.e[i]), y = to_f32(b.e[i]);
            a.e[i] = from_f32<T>(x * c[i] - y * s[i]);
            b.e[i] = from_f32<T>(y * c[i] + x * s[i]);
        }
    }
}

template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const T *x, T *y, const int32_t *__restrict__ pos, const double *__restrict__ inv_freq, int n_tok, int heads,
            int per_group, int D, int rot_begin, int rot_dim, long long xs, long long ys, float mscale, int inverse,
            int units) {
    const int n_rot = rot_dim / (2 * V);
    const long long e = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
    const int t = (int)(e / units);
    if (t >= n_tok) return;
    const int u = (int)(e - (long long)t * units);
    const RopeUnit<V, INTER> at(u, n_rot, rot_begin, rot_dim);
    float c[V], s[V];
    if (at.rot) {
        const int p = pos[t];
#pragma unroll
        for (int i = 0; i < V; ++i) rope_angle(p, inv_freq[u * V + i], mscale, inverse != 0, c[i], s[i]);
    }
    const int h0 = blockIdx.y * per_group, h1 = min(heads, h0 + per_group);
    for (int h = h0; h < h1; h += kRopeBatch) {
        Pack<T, V> a[kRopeBatch], b[kRopeBatch];
#pragma unroll
        for (int q = 0; q < kRopeBatch; ++q) {
            if (h + q < h1) {
                const T *row = x + t * xs + (long long)(h + q) * D;
                a[q].load(row + at.a);
                if (at.rot) b[q].load(row + at.b);
            }
        }
#pragma unroll
        for (int q = 0; q < kRopeBatch; ++q) {
            if (h + q < h1) {
                T *row = y + t * ys + (long long)(h + q) * D;
                if (at.rot) {
                    rope_turn<T, V, INTER>(a[q], b[q], c, s);
                    b[q].store(row + at.b);
                }
                a[q].store(row + at.a);
            }
        }
    }
}

// Heads per thread: all of them while the tokens alone fill the GPU (the angles are
// shared), fewer when there are few tokens.
inline int rope_groups(long long items, int heads, int sms) {
    const long long want = (long long)sms * 1536;
    long long g = items > 0 ? (want + items - 1) / items : 1;
    if (g < 1) g = 1;
    if (g > heads) g = heads;
    return (int)g;
}

template <typename T, int V>
int rope_launch(const crs_rope_params *p, int n_tok, int heads, const void *x, long long xs, const int32_t *pos,
                const double *inv_freq, void *y, long long ys, cudaStream_t s) {
    const int units = p->rot_dim / (2 * V) + (p->D - p->rot_dim) / V;
    const long long items = (long long)n_tok * units;
    const int per_group = ceil_div(heads, rope_groups(items, heads, cache_sms()));
    const dim3 grid((unsigned)ceil_div_ll(items, kRopeThreads), (unsigned)ceil_div(heads, per_group));
    ProfScope _ps(K_ROPE, s);
    if (p->interleaved)
        rope_kernel<T, V, true><<<grid, kRopeThreads, 0, s>>>(
            static_cast<const T *>(x), static_cast<T *>(y), pos, inv_freq, n_tok, heads, per_group, p->D, p->rot_begin,
            p->rot_dim, xs, ys, p->mscale, p->inverse, units);
    else
        rope_kernel<T, V, false><<<grid, kRopeThreads, 0, s>>>(
            static_cast<const T *>(x), static_cast<T *>(y), pos, inv_freq, n_tok, heads, per_group, p->D, p->rot_begin,
            p->rot_dim, xs, ys, p->mscale, p->inverse, units);
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
    int n_tok, n_q, rot_begin, rot_dim, units, per_group, inverse;
    float mscale;
};

// Heads are numbered k, v, q: a thread takes one vector of pairs of one token through
// its group of them.
template <bool INTER>
__global__ void __launch_bounds__(kRopeThreads) cache_append_kernel(AppendArgs a) {
    constexpr int V = 8;
    using P = Pack<__nv_bfloat16, V>;
    const long long e = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
    const long long tok = e / a.units;
    if (tok >= (long long)a.c.n_seq * a.n_tok) return;
    const int u = (int)(e - tok * a.units);
    const int s = (int)(tok / a.n_tok), i = (int)(tok - (long long)s * a.n_tok);
    const int n_kv = a.c.n_kv, D = a.c.D;
    const RopeUnit<V, INTER> at(u, a.rot_dim / (2 * V), a.rot_begin, a.rot_dim);
    const int hh0 = blockIdx.y * a.per_group, hh1 = min(2 * n_kv + a.n_q, hh0 + a.per_group);

    const int len = cache_len(a.c, s), n = cache_new(a.c, a.n_new, a.n_tok, s, len);
    const int asked = a.n_new ? min(max(a.n_new[s], 0), a.n_tok) : a.n_tok;
    const bool live = i < n;
    if (!live && i < asked && u == 0 && hh0 == 0) raise_error(CRS_DEVERR_CAPACITY);
    const int slot = len + i;
    const int position = a.c.next_pos[s] + i;
    const int row = live && hh0 < 2 * n_kv ? cache_row(a.c, s, slot) : -1;
    float c[V], sn[V];
    if (at.rot && live) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            rope_angle(position, a.inv_freq[u * V + j], a.mscale, a.inverse != 0, c[j], sn[j]);
    }
    for (int hh = hh0; hh < hh1; hh += kRopeBatch) {
        P x[kRopeBatch], y[kRopeBatch];
        __nv_bfloat16 *dst[kRopeBatch];
#pragma unroll
        for (int b = 0; b < kRopeBatch; ++b) {
            const int h = hh + b;
            dst[b] = nullptr;
            if (h >= hh1) continue;
            const __nv_bfloat16 *src;
            if (h < 2 * n_kv) {
                if (row < 0) continue;
                const bool is_k = h < n_kv;
                const int kh = is_k ? h : h - n_kv;
                src = (is_k ? a.k + tok * a.ks : a.v + tok * a.vs) + (size_t)kh * D;
                dst[b] = (is_k ? a.c.k : a.c.v) + ((size_t)row * n_kv + kh) * D;
                if (is_k && u == 0) {
                    const size_t m = ((size_t)s * n_kv + kh) * a.c.cap + slot;
                    if (a.c.pos) a.c.pos[m] = position;
                    if (a.c.mass) a.c.mass[m] = 0.0f;
                }
            } else {
                src = a.q + tok * a.qs + (size_t)(h - 2 * n_kv) * D;
                dst[b] = a.q_out + ((size_t)tok * a.n_q + (h - 2 * n_kv)) * D;
            }
            if (live) {
                x[b].load(src + at.a);
                if (at.rot) y[b].load(src + at.b);
            } else {
                x[b].w[0] = y[b].w[0] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
#pragma unroll
        for (int b = 0; b < kRopeBatch; ++b) {
            if (!dst[b]) continue;
            if (at.rot) {
                const int h = hh + b;
                if (live && (h < n_kv || h >= 2 * n_kv)) rope_turn<__nv_bfloat16, V, INTER>(x[b], y[b], c, sn);
                y[b].store(dst[b] + at.b);
            }
            x[b].store(dst[b] + at.a);
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
    if (ceil_div_ll((long long)n_tok * p->D, kRopeThreads) > 0x7fffffffLL) return CRS_ERR_UNSUPPORTED;
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
    a.units = a.rot_dim / 16 + (p->D - a.rot_dim) / 8;
    const int heads = 2 * p->n_kv + a.n_q;
    const long long items = (long long)p->n_seq * n_tok * a.units;
    if (ceil_div_ll(items, kRopeThreads) > 0x7fffffffLL || heads > 65535) return CRS_ERR_UNSUPPORTED;
    a.per_group = ceil_div(heads, rope_groups(items, heads, cache_sms()));
    const dim3 grid((unsigned)ceil_div_ll(items, kRopeThreads), (unsigned)ceil_div(heads, a.per_group));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    {
        ProfScope _ps(K_CACHE_APPEND, s);
        if (r && r->interleaved) cache_append_kernel<true><<<grid, kRopeThreads, 0, s>>>(a);
        else cache_append_kernel<false><<<grid, kRopeThreads, 0, s>>>(a);
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
