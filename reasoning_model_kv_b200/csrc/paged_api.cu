// paged_api.cu -- host side of the paged 8-bit cache's entry points: configuration and
// argument checks, the workspace's layout and the launches.
#include <climits>
#include <cmath>
#include <cstdio>
#include <new>
#include <string>

#include "paged.cuh"

struct tkv_paged {
    tkv_paged_config cfg;
    tkv::paged::View view;
    int64_t launches;
};

namespace tkv {
tkv_status api_fail(tkv_status st, const std::string &msg);
}

namespace {

using tkv::api_fail;
using tkv::paged::Rows;

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

const char *config_fault(const tkv_paged_config *c) {
    if (!c) return "config is NULL";
    if (c->B < 1 || c->B > 65535) return "B must be in [1, 65535]";
    if (c->Hkv < 1 || c->G < 1 || c->G > tkv::paged::kMaxGroup) return "Hkv must be >= 1 and G in [1, 16]";
    if ((long long)c->Hkv * c->G > 65535) return "Hkv * G must be <= 65535";
    if ((long long)c->B * c->Hkv > (1 << 24)) return "B * Hkv must be <= 2^24";
    if (c->D != 64 && c->D != 128) return "D must be 64 or 128";
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return "page must be 16, 32, 64 or 128";
    if (c->pages < 1 || c->max_pages < 1) return "pages and max_pages must be >= 1";
    if ((long long)c->max_pages * c->page > (1ll << 30)) return "max_pages * page must be <= 2^30";
    if ((long long)c->pages * c->Hkv > INT_MAX) return "pages * Hkv must be < 2^31";
    if (c->code != TKV_CODE_INT8 && c->code != TKV_CODE_E4M3) return "code must be TKV_CODE_INT8 or TKV_CODE_E4M3";
    if (c->dtype != TKV_DTYPE_BF16 && c->dtype != TKV_DTYPE_FP16) return "dtype must be TKV_DTYPE_BF16 or TKV_DTYPE_FP16";
    return nullptr;
}

const char *rope_fault(const tkv_rope *r, int D) {
    if (r->rot < 0 || r->rot > D || r->rot % 8) return "rot must be a multiple of 8 in [0, D]";
    if (r->rot > 0 && (!r->inv_freq || !aligned(r->inv_freq, 4))) return "inv_freq is NULL or not 4-byte aligned";
    if (r->interleaved != 0 && r->interleaved != 1) return "interleaved must be 0 or 1";
    if ((r->q_weight == nullptr) != (r->k_weight == nullptr)) return "q_weight and k_weight: both or none";
    if (!aligned(r->q_weight, 2) || !aligned(r->k_weight, 2)) return "weights must be 2-byte aligned";
    if (r->q_weight && !(r->eps >= 0.f && std::isfinite(r->eps))) return "eps must be finite and >= 0";
    return nullptr;
}

Rows rows(const tkv_rows &r) { return {r.p, (long long)r.token_stride, (long long)r.head_stride}; }

// Rows of one call: pointers and strides that eight-byte accesses can use.
const char *rows_fault(const Rows &r) {
    if (!r.p) return "NULL row array";
    if (!aligned(r.p, 8)) return "row arrays must be 8-byte aligned";
    if (r.token % 4 || r.head % 4) return "row strides must be multiples of 4 elements";
    if (r.token < 0 || r.head < 0) return "row strides must be >= 0";
    return nullptr;
}
const char *out_fault(const Rows &r, int T, int heads, int D) {
    if (const char *w = rows_fault(r)) return w;
    // rows that overlap would be written by several threads: a token's heads lie within its stride, or
    // a head's tokens within that one's
    if ((heads > 1 && r.head < D) || (T > 1 && r.token < D)) return "output rows overlap";
    if (heads > 1 && T > 1 && heads - 1 > (r.token - D) / r.head && T - 1 > (r.head - D) / r.token)
        return "output rows overlap";
    return nullptr;
}

tkv_status cuda_status(cudaError_t e, const char *what) {
    if (e == cudaSuccess) return TKV_OK;
    return api_fail(TKV_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

tkv_status bad(const char *why) { return api_fail(TKV_ERR_INVALID, why); }

const char *lengths_fault(const tkv_paged *c, const int32_t *table, const int32_t *len, const int32_t *cu, int T) {
    if (!table || !len) return "NULL block_table or kv_len";
    if (!aligned(table, 4) || !aligned(len, 4) || !aligned(cu, 4)) return "int32 arrays must be 4-byte aligned";
    if (T < 0 || T > tkv::paged::kMaxLen) return "T must be in [0, 2^30]";
    if (!cu && T != c->cfg.B) return "without cu, T must be B";
    return nullptr;
}

}  // namespace

namespace tkv {
namespace paged {
size_t attention_workspace_bytes(const tkv_paged_config &cfg);
size_t attention_reset_bytes();      // at the workspace's start, behind the error word
}
}  // namespace tkv

extern "C" {

tkv_status tkv_qk_norm_rope(const tkv_qk_norm_rope_args *a, void *stream) {
    if (!a || !a->rope) return bad("args or rope is NULL");
    const int T = a->T, Hq = a->Hq, Hkv = a->Hkv, D = a->D;
    if (D != 64 && D != 128) return bad("D must be 64 or 128");
    if (a->dtype != TKV_DTYPE_BF16 && a->dtype != TKV_DTYPE_FP16)
        return bad("dtype must be TKV_DTYPE_BF16 or TKV_DTYPE_FP16");
    if (T < 0 || Hq < 0 || Hkv < 0 || Hq > 65535 || Hkv > 65535) return bad("T, Hq or Hkv out of range");
    if (const char *w = rope_fault(a->rope, D)) return bad(w);
    if (T == 0 || Hq + Hkv == 0) return TKV_OK;
    if (!a->pos || !aligned(a->pos, 4)) return bad("pos is NULL or not 4-byte aligned");
    const Rows q = rows(a->q), k = rows(a->k), qo = rows(a->q_out), ko = rows(a->k_out);
    if (Hq > 0) {
        if (const char *w = rows_fault(q)) return bad(w);
        if (const char *w = out_fault(qo, T, Hq, D)) return bad(w);
    }
    if (Hkv > 0) {
        if (const char *w = rows_fault(k)) return bad(w);
        if (const char *w = out_fault(ko, T, Hkv, D)) return bad(w);
    }
    return cuda_status(tkv::paged::launch_norm_rope(*a->rope, q, k, a->pos, qo, ko, T, Hq, Hkv, D, a->dtype,
                                                    static_cast<cudaStream_t>(stream)),
                       "tkv_qk_norm_rope");
}

size_t tkv_paged_workspace_bytes(const tkv_paged_config *cfg) {
    if (const char *w = config_fault(cfg)) { api_fail(TKV_ERR_INVALID, w); return 0; }
    return 256 + tkv::paged::attention_workspace_bytes(*cfg);
}

tkv_status tkv_paged_create(const tkv_paged_config *cfg, void *k_pool, void *v_pool, float *k_scale, float *v_scale,
                            void *d_workspace, size_t workspace_bytes, tkv_paged **out) {
    if (!out) return bad("out is NULL");
    *out = nullptr;
    if (const char *w = config_fault(cfg)) return bad(w);
    if (!k_pool || !v_pool || !k_scale || !v_scale) return bad("NULL pool or scale pointer");
    if (!aligned(k_pool, 16) || !aligned(v_pool, 16)) return bad("pools must be 16-byte aligned");
    if (!aligned(k_scale, 4) || !aligned(v_scale, 4)) return bad("scales must be 4-byte aligned");
    if (!d_workspace || !aligned(d_workspace, 256)) return bad("workspace must be 256-byte aligned and not NULL");
    if (workspace_bytes < tkv_paged_workspace_bytes(cfg)) return bad("workspace too small");
    auto *c = new (std::nothrow) tkv_paged();
    if (!c) return bad("out of host memory");
    c->cfg = *cfg;
    c->launches = 0;
    int lg = 0;
    while ((1 << lg) < cfg->page) ++lg;
    c->view = {cfg->B, cfg->Hkv, cfg->G, cfg->D, cfg->page, lg, cfg->pages, cfg->max_pages, cfg->code, cfg->dtype,
               static_cast<uint8_t *>(k_pool), static_cast<uint8_t *>(v_pool), k_scale, v_scale,
               static_cast<uint32_t *>(d_workspace)};
    *out = c;
    return TKV_OK;
}

tkv_status tkv_paged_destroy(tkv_paged *c) {
    delete c;
    return TKV_OK;
}

tkv_status tkv_paged_reset(tkv_paged *c, void *stream) {
    if (!c) return bad("cache is NULL");
    return cuda_status(cudaMemsetAsync(c->view.err, 0, 256 + tkv::paged::attention_reset_bytes(), static_cast<cudaStream_t>(stream)), "tkv_paged_reset");
}

tkv_status tkv_paged_append(tkv_paged *c, const tkv_paged_append_args *a, void *stream) {
    if (!c || !a) return bad("cache or args is NULL");
    const int T = a->T;
    if (const char *w = lengths_fault(c, a->block_table, a->kv_len, a->cu, T)) return bad(w);
    const tkv_rope none{};
    const tkv_rope &r = a->rope ? *a->rope : none;
    if (const char *w = rope_fault(&r, c->cfg.D)) return bad(w);
    if (a->max_new < 1 || a->max_new > tkv::paged::kMaxLen) return bad("max_new must be in [1, 2^30]");
    if (T == 0) return TKV_OK;
    const Rows k = rows(a->k), v = rows(a->v), q = rows(a->q), qo = rows(a->q_out);
    if (const char *w = rows_fault(k)) return bad(w);
    if (const char *w = rows_fault(v)) return bad(w);
    if (q.p) {
        if (const char *w = rows_fault(q)) return bad(w);
        if (const char *w = out_fault(qo, T, c->cfg.Hkv * c->cfg.G, c->cfg.D)) return bad(w);
    } else if (qo.p) {
        return bad("q_out without q");
    }
    return cuda_status(tkv::paged::launch_append(c->view, r, k, v, q, qo, T, a->block_table, a->kv_len, a->cu,
                                                 a->max_new < T ? a->max_new : T, static_cast<cudaStream_t>(stream),
                                                 &c->launches),
                       "tkv_paged_append");
}

tkv_status tkv_paged_attention(tkv_paged *c, const tkv_paged_attention_args *a, void *stream) {
    if (!c || !a) return bad("cache or args is NULL");
    const int T = a->T;
    if (const char *w = lengths_fault(c, a->block_table, a->kv_len, a->cu, T)) return bad(w);
    if (a->max_q < 1) return bad("max_q must be >= 1");
    if (a->window < 0) return bad("window must be >= 0");
    if (!std::isfinite(a->softmax_scale * tkv::paged::kLog2e)) return bad("softmax_scale must be finite, in units of log2 too");
    if (T == 0) return TKV_OK;
    const Rows q = rows(a->q), out = rows(a->out);
    if (const char *w = rows_fault(q)) return bad(w);
    if (const char *w = out_fault(out, T, c->cfg.Hkv * c->cfg.G, c->cfg.D)) return bad(w);
    return cuda_status(tkv::paged::launch_attention(c->view, q, out, T, a->block_table, a->kv_len, a->cu, a->max_q,
                                                    a->window, a->softmax_scale, static_cast<cudaStream_t>(stream),
                                                    &c->launches),
                       "tkv_paged_attention");
}

tkv_status tkv_paged_poll_error(tkv_paged *c, void *stream) {
    if (!c) return bad("cache is NULL");
    auto st = static_cast<cudaStream_t>(stream);
    uint32_t w[4] = {0, 0, 0, 0};
    cudaError_t e = cudaMemcpyAsync(w, c->view.err, sizeof(w), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e == cudaSuccess) e = cudaMemsetAsync(c->view.err, 0, sizeof(w), st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_status(e, "tkv_paged_poll_error");
    if (w[0] == 0) return TKV_OK;
    char msg[160];
    std::snprintf(msg, sizeof(msg), "device error %u (%u occurrences, detail %u)", w[0], w[1], w[2]);
    return api_fail(static_cast<tkv_status>(w[0]), msg);
}

int64_t tkv_paged_launch_count(const tkv_paged *c) { return c ? c->launches : 0; }

}  // extern "C"
