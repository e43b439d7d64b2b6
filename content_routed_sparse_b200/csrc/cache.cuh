// What the kernels of the paged decode cache share: its state on the device, slot
// addresses, and the host checks (sm_100a).
#pragma once

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

// SM count of the current device (148 where it cannot be read: the sizing stays valid).
inline int cache_sms() {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        sms = 148;
    }
    return sms;
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
    int PT;            // key tiles of a prefix item of cache_attn_kernel (0: none)
    int PRT;           // its row tiles, over n_seq * M rows
    int grid;          // CTAs of cache_attn_kernel
    int tc_splits;     // key splits of cache_prefix_kernel (0: not launched)
    int tc_tiles;      // its row tiles per KV head, kPfRows rows each
    float scale_log2, decay;
    float *part_o, *part_ml;       // pieces: [piece][16][D], [piece][16][2] (m in log2 units, l)
    float *tc_o, *tc_ml;           // [split][KV head][n_seq * M][D], [..][2]
    float *logits;                 // [sequence][KV head][M][ls] log2-scaled, or null
    int ls;
    void *O;
    float *lse, *mass_out;
};

}  // namespace crs
