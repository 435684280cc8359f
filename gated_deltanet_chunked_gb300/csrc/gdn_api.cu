// C ABI of libgdn.so: argument checks, workspace carving and dispatch.
//
// Every entry point validates all of its arguments before the first launch
// and returns a gdn_status; nothing is enqueued on failure. There is one
// compute path per io dtype (f32: SIMT kernels; bf16: tensor-core kernels)
// and no host-side fallback of any kind.
#include <atomic>
#include <initializer_list>
#include <mutex>

#include "gdn_common.cuh"
#include "gdn_linrec.cuh"
#include "tma_host.cuh"

namespace gdn {
namespace {

__device__ int g_status_word;  // device status word (first device-side error)

constexpr unsigned long long kDefaultWaitNs = 2000000000ull;
std::atomic<unsigned long long> g_wait_ns{kDefaultWaitNs};  // limit of bounded waits

constexpr int kMaxDevices = 64;
int *g_status_ptr[kMaxDevices];
unsigned long long g_status_ctx[kMaxDevices];  // context id the cached address belongs to
std::mutex g_status_mu;

// Device address of the status word for the current device, looked up once
// per device and context (cudaGetSymbolAddress needs that device current;
// the context id catches a cudaDeviceReset, after which the module and its
// variables are loaded anew).
int *status_ptr() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lk(g_status_mu);
    unsigned long long ctx = 0;
    const bool have_ctx = current_context_id(&ctx);
    if (!g_status_ptr[dev] || !have_ctx || g_status_ctx[dev] != ctx) {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_status_word) != cudaSuccess) return nullptr;
        g_status_ptr[dev] = static_cast<int *>(p);
        // the symbol lookup made the context current if it was not yet
        g_status_ctx[dev] = (have_ctx || current_context_id(&ctx)) ? ctx : 0;
    }
    return g_status_ptr[dev];
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Checks shared by prefill and decode. Returns GDN_OK or the error code.
// `allowed_flags`: the gdn_problem.flags bits the entry point accepts.
int check_common(const gdn_problem *p, uint32_t allowed_flags = 0) {
    if (!p) return GDN_EINVAL;
    if (p->hq <= 0 || p->hv <= 0 || p->dk <= 0 || p->dv <= 0) return GDN_EINVAL;
    if (p->hv % p->hq != 0) return GDN_EINVAL;
    if (p->io_dtype != GDN_DT_F32 && p->io_dtype != GDN_DT_BF16) return GDN_EINVAL;
    if (p->num_seqs < 0 || p->total_tokens < 0) return GDN_EINVAL;
    if (p->dk != kHeadDim || p->dv != kHeadDim) return GDN_EUNSUPPORTED;
    if (p->flags & ~allowed_flags) return GDN_EUNSUPPORTED;
    return GDN_OK;
}

int check_prefill_shape(const gdn_problem *p, bool packed) {
    int st = check_common(p);
    if (st) return st;
    if (p->num_seqs < 1) return GDN_EINVAL;
    if (!packed) {
        if (p->batch < 1 || p->seqlen < 0 || p->num_seqs != p->batch) return GDN_EINVAL;
        if (int64_t(p->batch) * p->seqlen != p->total_tokens) return GDN_EINVAL;
    }
    // token-row products must stay addressable with 64-bit offsets and the
    // chunk count must fit the int32 chunk table
    if (int64_t(p->total_tokens) / kChunk + p->num_seqs > (int64_t(1) << 30)) return GDN_EINVAL;
    // the per-(chunk, head) flags and counters are indexed with int
    if ((int64_t(p->total_tokens) / kChunk + p->num_seqs) * p->hv * 2 >= (int64_t(1) << 31)) return GDN_EINVAL;
    return GDN_OK;
}

int max_chunks_of(const gdn_problem *p) { return p->total_tokens / kChunk + p->num_seqs; }

// Workspace layout: [n_chunks | seq_info | chunk_info | kernel data].
struct WsLayout {
    size_t seq_off, chunk_off, data_off, data_bytes, total;
};

WsLayout ws_layout(const gdn_problem *p) {
    WsLayout l;
    const int mc = max_chunks_of(p);
    l.seq_off = 256;
    l.chunk_off = l.seq_off + align256(sizeof(SeqInfo) * size_t(p->num_seqs));
    l.data_off = l.chunk_off + align256(sizeof(ChunkInfo) * size_t(mc));
    l.data_bytes = p->io_dtype == GDN_DT_BF16 ? prefill_tc_workspace(mc, p->hv) : prefill_simt_workspace(mc, p->hv);
    l.total = l.data_off + l.data_bytes;
    return l;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ECUDA; }

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_version(void) { return 103; }

const char *gdn_status_string(int status) {
    switch (status) {
        case GDN_OK: return "GDN_OK";
        case GDN_EINVAL: return "GDN_EINVAL: invalid argument (pointer, shape, size or alignment)";
        case GDN_EUNSUPPORTED: return "GDN_EUNSUPPORTED: valid but unsupported (dk/dv must be 128, flags 0)";
        case GDN_ECUDA: return "GDN_ECUDA: a CUDA runtime call or kernel launch failed";
        case GDN_ETIMEOUT: return "GDN_ETIMEOUT: a bounded device-side wait gave up";
        case GDN_EDEVICE_INPUT: return "GDN_EDEVICE_INPUT: device-side input check failed (cu_seqlens or slot index)";
        case GDN_ETOOBIG:
            return "GDN_ETOOBIG: workspace need exceeds the fixed no-alloc scratch (GDN_NOALLOC_SCRATCH_BYTES)";
        default: return "unknown gdn_status";
    }
}

size_t gdn_chunk_fwd_workspace_size(const gdn_problem *p) {
    // the size depends only on total_tokens, num_seqs and hv, so the packed
    // checks (a superset of nothing layout-specific) are the right ones here
    if (check_prefill_shape(p, /*packed=*/true) != GDN_OK) return 0;
    return ws_layout(p).total;
}

}  // extern "C"

namespace gdn {
namespace {

// The output gate of gdn_chunk_fwd_gated (null z: none).
struct OutGate {
    const void *z;
    const float *weight;
    float eps;
};

int chunk_fwd(const gdn_problem *p, const void *q, const void *k, const void *v, const float *g, const float *beta,
              float scale, const float *initial_state, const int32_t *cu_seqlens, const OutGate &gate, void *out,
              float *final_state, void *workspace, size_t workspace_bytes, void *stream) {
    const bool packed = cu_seqlens != nullptr;
    int st = check_prefill_shape(p, packed);
    if (st) return st;
    if (p->total_tokens > 0) {
        if (!q || !k || !v || !g || !beta || !out) return GDN_EINVAL;
        if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta) || !aligned16(out))
            return GDN_EINVAL;
    }
    if ((initial_state && !aligned16(initial_state)) || (final_state && !aligned16(final_state)) ||
        (cu_seqlens && !aligned16(cu_seqlens)))
        return GDN_EINVAL;
    const WsLayout L = ws_layout(p);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < L.total)
        return GDN_EINVAL;
    int *status = status_ptr();
    if (!status) return GDN_ECUDA;

    char *ws = static_cast<char *>(workspace);
    PrefillArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
    a.s0 = initial_state; a.final_state = final_state; a.out = out; a.scale = scale;
    a.hq = p->hq; a.hv = p->hv; a.group = p->hv / p->hq;
    a.num_seqs = p->num_seqs; a.total_tokens = p->total_tokens;
    a.dense_batch = packed ? 0 : p->batch;
    a.dense_seqlen = packed ? 0 : p->seqlen;
    a.cu = cu_seqlens;
    a.max_chunks = max_chunks_of(p);
    a.n_chunks = reinterpret_cast<int *>(ws);
    a.seq_info = reinterpret_cast<SeqInfo *>(ws + L.seq_off);
    a.chunk_info = reinterpret_cast<ChunkInfo *>(ws + L.chunk_off);
    a.status = status;
    a.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
    if (p->io_dtype == GDN_DT_BF16) {
        a.ready = prefill_tc_ready_flags(ws + L.data_off, a.max_chunks, a.hv);
        a.done = a.ready + size_t(a.max_chunks) * a.hv;  // output counters follow the ready flags
        a.ready_count = 2 * a.max_chunks * a.hv;
    }
    if (gate.z) {
        if (p->total_tokens > 0 && (!aligned16(gate.z) || !gate.weight || !aligned16(gate.weight))) return GDN_EINVAL;
        if (!(gate.eps >= 0.f)) return GDN_EINVAL;
        a.z = gate.z;
        a.norm_weight = gate.weight;
        a.norm_eps = gate.eps;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = cuda_status(launch_chunk_table(a, s)))) return st;
    if (p->io_dtype == GDN_DT_BF16) return cuda_status(launch_prefill_tc(a, ws + L.data_off, s));
    if ((st = cuda_status(launch_prefill_simt(a, ws + L.data_off, s)))) return st;
    if (!gate.z) return GDN_OK;
    return cuda_status(launch_gated_rmsnorm(out, gate.z, gate.weight, gate.eps, out,
                                            (long long)p->total_tokens * p->hv, p->io_dtype, status, s));
}

}  // namespace
}  // namespace gdn

extern "C" {

int gdn_chunk_fwd(const gdn_problem *p, const void *q, const void *k, const void *v, const float *g,
                  const float *beta, float scale, const float *initial_state, const int32_t *cu_seqlens,
                  void *out, float *final_state, void *workspace, size_t workspace_bytes, void *stream) {
    return gdn::chunk_fwd(p, q, k, v, g, beta, scale, initial_state, cu_seqlens, gdn::OutGate{nullptr, nullptr, 0.f},
                          out, final_state, workspace, workspace_bytes, stream);
}

int gdn_chunk_fwd_gated(const gdn_problem *p, const void *q, const void *k, const void *v, const float *g,
                        const float *beta, float scale, const float *initial_state, const int32_t *cu_seqlens,
                        const void *z, const float *norm_weight, float norm_eps, void *out, float *final_state,
                        void *workspace, size_t workspace_bytes, void *stream) {
    if (!z) return GDN_EINVAL;
    return gdn::chunk_fwd(p, q, k, v, g, beta, scale, initial_state, cu_seqlens,
                          gdn::OutGate{z, norm_weight, norm_eps}, out, final_state, workspace, workspace_bytes,
                          stream);
}

constexpr uint32_t kDecodeFlags = GDN_FLAG_BETA_BF16 | GDN_FLAG_STATE_BF16;

int gdn_recurrent_step(const gdn_problem *p, const void *q, const void *k, const void *v, const float *g,
                       const float *beta, float scale, void *state, const int32_t *state_indices, void *out,
                       void *stream) {
    int st = check_common(p, kDecodeFlags);
    if (st) return st;
    if (p->total_tokens != p->num_seqs) return GDN_EINVAL;
    if (p->num_state_slots < 0 || (!state_indices && p->num_state_slots < p->num_seqs)) return GDN_EINVAL;
    if (p->num_seqs > 0) {
        if (!q || !k || !v || !g || !beta || !out || !state) return GDN_EINVAL;
        if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta) ||
            !aligned16(out) || !aligned16(state) || (state_indices && !aligned16(state_indices)))
            return GDN_EINVAL;
    }
    if (int64_t(p->num_seqs) * p->hv >= (int64_t(1) << 31)) return GDN_EINVAL;
    int *status = status_ptr();
    if (!status) return GDN_ECUDA;
    return cuda_status(launch_recurrent_step(*p, q, k, v, g, beta, nullptr, scale, state, state_indices, out,
                                             status, static_cast<cudaStream_t>(stream)));
}

int gdn_recurrent_step_gated(const gdn_problem *p, const void *q, const void *k, const void *v, const float *a,
                             const float *b, const float *A_log, const float *dt_bias, float scale, void *state,
                             const int32_t *state_indices, const void *z, const float *norm_weight,
                             float norm_eps, void *out, void *stream) {
    int st = check_common(p, kDecodeFlags);
    if (st) return st;
    if (p->total_tokens != p->num_seqs) return GDN_EINVAL;
    if (p->num_state_slots < 0 || (!state_indices && p->num_state_slots < p->num_seqs)) return GDN_EINVAL;
    if (p->num_seqs > 0) {
        if (!q || !k || !v || !a || !b || !A_log || !dt_bias || !out || !state) return GDN_EINVAL;
        if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(state) ||
            (state_indices && !aligned16(state_indices)))
            return GDN_EINVAL;
        if (!aligned4(a) || !aligned4(b) || !aligned4(A_log) || !aligned4(dt_bias)) return GDN_EINVAL;
        if (z && (!norm_weight || !aligned16(z) || !aligned16(norm_weight))) return GDN_EINVAL;
    }
    if (z && !(norm_eps >= 0.f)) return GDN_EINVAL;
    if (int64_t(p->num_seqs) * p->hv >= (int64_t(1) << 31)) return GDN_EINVAL;
    int *status = status_ptr();
    if (!status) return GDN_ECUDA;
    const DecodeFront front{a, b, A_log, dt_bias, z, z ? norm_weight : nullptr, norm_eps};
    return cuda_status(launch_recurrent_step(*p, q, k, v, nullptr, nullptr, &front, scale, state, state_indices,
                                             out, status, static_cast<cudaStream_t>(stream)));
}

int gdn_gated_rmsnorm(const gdn_problem *p, const void *o, const void *z, const float *weight, float eps, void *y,
                      void *stream) {
    if (!p || p->hv <= 0 || p->total_tokens < 0) return GDN_EINVAL;
    if (p->io_dtype != GDN_DT_F32 && p->io_dtype != GDN_DT_BF16) return GDN_EINVAL;
    if (p->dv != kHeadDim) return p->dv > 0 ? GDN_EUNSUPPORTED : GDN_EINVAL;
    if (!(eps >= 0.f)) return GDN_EINVAL;
    const long long rows = (long long)p->total_tokens * p->hv;
    if (rows > 0) {
        if (!o || !z || !weight || !y) return GDN_EINVAL;
        if (!aligned16(o) || !aligned16(z) || !aligned16(weight) || !aligned16(y)) return GDN_EINVAL;
    }
    int *status = status_ptr();
    if (!status) return GDN_ECUDA;
    return cuda_status(launch_gated_rmsnorm(o, z, weight, eps, y, rows, p->io_dtype, status,
                                            static_cast<cudaStream_t>(stream)));
}

int gdn_causal_conv1d_silu(const gdn_problem *p, const void *x, const float *weight, const float *bias,
                           void *conv_state, const int32_t *state_indices, const int32_t *cu_seqlens, int norm_qk,
                           void *q, void *k, void *v, void *stream) {
    int st = check_common(p);
    if (st) return st;
    if (p->num_seqs < 1 || p->num_state_slots < 0) return GDN_EINVAL;
    if (!cu_seqlens && p->num_seqs != 1) return GDN_EINVAL;
    if (conv_state && !state_indices && p->num_state_slots < p->num_seqs) return GDN_EINVAL;
    // token offsets stay in int (a tile start plus its length), channel blocks in grid.y
    if (int64_t(p->total_tokens) + 64 >= (int64_t(1) << 31) || (2 * p->hq + p->hv) > 65535 * 8) return GDN_EINVAL;
    if (!weight || !aligned16(weight) || (bias && !aligned16(bias))) return GDN_EINVAL;
    if ((conv_state && !aligned16(conv_state)) || (state_indices && !aligned4(state_indices)) ||
        (cu_seqlens && !aligned4(cu_seqlens)))
        return GDN_EINVAL;
    if (p->total_tokens > 0) {
        if (!x || !q || !k || !v) return GDN_EINVAL;
        if (!aligned16(x) || !aligned16(q) || !aligned16(k) || !aligned16(v)) return GDN_EINVAL;
    }
    int *status = status_ptr();
    if (!status) return GDN_ECUDA;
    return cuda_status(launch_conv1d_silu(*p, x, weight, bias, conv_state, state_indices, cu_seqlens, norm_qk, q, k,
                                          v, status, static_cast<cudaStream_t>(stream)));
}

int gdn_causal_conv1d_silu_step(const gdn_problem *p, const void *x, const float *weight, const float *bias,
                                void *conv_state, const int32_t *state_indices, int norm_qk, void *q, void *k,
                                void *v, void *stream) {
    int st = check_common(p);
    if (st) return st;
    if (p->num_seqs < 0 || p->total_tokens != p->num_seqs || p->num_state_slots < 0) return GDN_EINVAL;
    if (conv_state && !state_indices && p->num_state_slots < p->num_seqs) return GDN_EINVAL;
    if ((2 * p->hq + p->hv) > 65535 * 8) return GDN_EINVAL;
    if (!weight || !aligned16(weight) || (bias && !aligned16(bias))) return GDN_EINVAL;
    if ((conv_state && !aligned16(conv_state)) || (state_indices && !aligned4(state_indices))) return GDN_EINVAL;
    if (p->num_seqs > 0) {
        if (!x || !q || !k || !v) return GDN_EINVAL;
        if (!aligned16(x) || !aligned16(q) || !aligned16(k) || !aligned16(v)) return GDN_EINVAL;
    }
    int *status = status_ptr();
    if (!status) return GDN_ECUDA;
    return cuda_status(launch_conv1d_step(*p, x, weight, bias, conv_state, state_indices, norm_qk, q, k, v, status,
                                          static_cast<cudaStream_t>(stream)));
}

int gdn_gating(const gdn_problem *p, const float *a, const float *b, const float *A_log, const float *dt_bias,
               float *g, float *beta, void *stream) {
    if (!p || p->hv <= 0 || p->total_tokens < 0) return GDN_EINVAL;
    const long long n = (long long)p->total_tokens * p->hv;
    if (n > 0) {
        if (!a || !b || !A_log || !dt_bias || !g || !beta) return GDN_EINVAL;
        if (!aligned4(a) || !aligned4(b) || !aligned4(A_log) || !aligned4(dt_bias) || !aligned4(g) ||
            !aligned4(beta))
            return GDN_EINVAL;
    }
    return cuda_status(launch_gating(a, b, A_log, dt_bias, g, beta, n, p->hv, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace gdn {
namespace {

struct Span {
    const void *p;
    size_t bytes;
};

bool overlap(const Span &a, const Span &b) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.p), q = reinterpret_cast<uintptr_t>(b.p);
    return p && q && a.bytes && b.bytes && p < q + b.bytes && q < p + a.bytes;
}

// Whether an output overlaps an input or another output. The first `in_place`
// outputs may be any of the first `as` inputs, in exactly its place.
bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins, int in_place = 0, int as = 0) {
    int o = 0;
    for (auto a = outs.begin(); a != outs.end(); ++a, ++o) {
        for (auto b = a + 1; b != outs.end(); ++b)
            if (overlap(*a, *b)) return true;
        int i = 0;
        for (const Span &b : ins) {
            const bool may = o < in_place && i++ < as && a->p == b.p;
            if (!may && overlap(*a, b)) return true;
        }
    }
    return false;
}

size_t io_bytes(const gdn_problem *p, size_t elements) { return elements * (p->io_dtype == GDN_DT_BF16 ? 2 : 4); }

// Descriptor checks of the gated linear recurrence's forward and backward pass.
int check_linrec(const gdn_problem *p, bool packed) {
    if (!p || p->hv <= 0 || p->dv <= 0 || p->num_seqs < 1 || p->total_tokens < 0) return GDN_EINVAL;
    if (p->io_dtype != GDN_DT_F32 && p->io_dtype != GDN_DT_BF16) return GDN_EINVAL;
    if (p->dv != kHeadDim || (p->flags & ~uint32_t(GDN_FLAG_GATE_CHANNEL))) return GDN_EUNSUPPORTED;
    if (!packed) {
        if (p->batch < 1 || p->seqlen < 0 || p->num_seqs != p->batch) return GDN_EINVAL;
        if (int64_t(p->batch) * p->seqlen != p->total_tokens) return GDN_EINVAL;
    }
    // token indices a few tiles past the end, a row's bytes and the number of CTAs stay in 32 bits
    if (p->total_tokens > INT32_MAX - 65536 || p->hv > (1 << 20) || p->num_seqs == INT32_MAX) return GDN_EINVAL;
    return GDN_OK;
}

// g and dg: per channel like x, or f32 per head
bool gate_ok(const gdn_problem *p, const void *g) {
    return g && (p->flags & GDN_FLAG_GATE_CHANNEL ? aligned16(g) : aligned4(g));
}

// the recurrence's tensors: rows [total_tokens, hv, 128], gates, states [seqs, hv, 128], offsets
Span rows_of(const gdn_problem *p, const void *x) {
    return {x, io_bytes(p, size_t(p->total_tokens) * p->hv * kHeadDim)};
}
Span gates_of(const gdn_problem *p, const void *g) {
    return p->flags & GDN_FLAG_GATE_CHANNEL ? rows_of(p, g) : Span{g, size_t(p->total_tokens) * p->hv * sizeof(float)};
}
Span states_of(const gdn_problem *p, const void *s, size_t seqs) {
    return {s, seqs * p->hv * kHeadDim * sizeof(float)};
}
Span offsets_of(const gdn_problem *p, const void *cu) { return {cu, (size_t(p->num_seqs) + 1) * sizeof(int32_t)}; }

RecArgs linrec_args(const gdn_problem *p, const void *x, const void *g, const float *s0, const int32_t *cu) {
    RecArgs a{};
    a.x = x; a.g = g; a.s0 = s0; a.cu = cu;
    a.total_tokens = p->total_tokens; a.num_seqs = p->num_seqs; a.hv = p->hv;
    a.dense_seqlen = cu ? 0 : p->seqlen;
    a.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
    return a;
}

}  // namespace
}  // namespace gdn

extern "C" {

size_t gdn_linear_recurrence_states_size(const gdn_problem *p) {
    if (check_linrec(p, /*packed=*/true) != GDN_OK) return 0;  // the size does not depend on the layout
    return (size_t(p->total_tokens) + kStateRows - 1) / kStateRows * size_t(p->hv) * kHeadDim * sizeof(float);
}

int gdn_linear_recurrence(const gdn_problem *p, const void *x, const void *g, const float *initial_state,
                          const int32_t *cu_seqlens, void *out, float *final_state, float *states, void *stream) {
    int st = check_linrec(p, cu_seqlens != nullptr);
    if (st) return st;
    if (p->total_tokens > 0 && (!x || !out || !aligned16(x) || !aligned16(out) || !gate_ok(p, g)))
        return GDN_EINVAL;
    if (!aligned16(initial_state) || !aligned4(cu_seqlens) || !aligned16(final_state) || !aligned16(states))
        return GDN_EINVAL;
    const size_t seqs = size_t(p->num_seqs);
    if (clash({rows_of(p, out), states_of(p, final_state, seqs), {states, gdn_linear_recurrence_states_size(p)}},
              {rows_of(p, x), gates_of(p, g), states_of(p, initial_state, seqs), offsets_of(p, cu_seqlens)}))
        return GDN_EINVAL;
    RecArgs a = linrec_args(p, x, g, initial_state, cu_seqlens);
    a.out = out; a.final_state = final_state; a.states = states;
    if (!(a.status = status_ptr())) return GDN_ECUDA;
    return cuda_status(launch_linrec(a, p->io_dtype, p->flags & GDN_FLAG_GATE_CHANNEL,
                                     static_cast<cudaStream_t>(stream)));
}

int gdn_linear_recurrence_bwd(const gdn_problem *p, const void *dout, const void *x, const void *g,
                              const float *states, const float *initial_state, const float *dfinal_state,
                              const int32_t *cu_seqlens, void *dx, void *dg, float *dinitial_state, void *stream) {
    int st = check_linrec(p, cu_seqlens != nullptr);
    if (st) return st;
    if (p->total_tokens > 0) {
        if (!dout || !x || !states || !dx || !gate_ok(p, g) || !gate_ok(p, dg)) return GDN_EINVAL;
        if (!aligned16(dout) || !aligned16(x) || !aligned16(states) || !aligned16(dx)) return GDN_EINVAL;
    }
    if (!aligned16(initial_state) || !aligned16(dfinal_state) || !aligned4(cu_seqlens) || !aligned16(dinitial_state))
        return GDN_EINVAL;
    const size_t seqs = size_t(p->num_seqs);
    if (clash({rows_of(p, dx), gates_of(p, dg), states_of(p, dinitial_state, seqs)},
              {rows_of(p, dout), rows_of(p, x), gates_of(p, g), {states, gdn_linear_recurrence_states_size(p)},
               states_of(p, initial_state, seqs), states_of(p, dfinal_state, seqs), offsets_of(p, cu_seqlens)}))
        return GDN_EINVAL;
    RecArgs a = linrec_args(p, x, g, initial_state, cu_seqlens);
    a.dout = dout; a.dfinal = dfinal_state; a.dx = dx; a.dg = dg; a.dinitial = dinitial_state;
    a.states = const_cast<float *>(states);  // read only
    if (!(a.status = status_ptr())) return GDN_ECUDA;
    return cuda_status(launch_linrec_bwd(a, p->io_dtype, p->flags & GDN_FLAG_GATE_CHANNEL,
                                         static_cast<cudaStream_t>(stream)));
}

int gdn_linear_recurrence_step(const gdn_problem *p, const void *x, const void *g, float *state,
                               const int32_t *state_indices, void *out, void *stream) {
    if (!p || p->hv <= 0 || p->dv <= 0 || p->num_seqs < 0 || p->total_tokens != p->num_seqs) return GDN_EINVAL;
    if (p->io_dtype != GDN_DT_F32 && p->io_dtype != GDN_DT_BF16) return GDN_EINVAL;
    if (p->dv != kHeadDim || (p->flags & ~uint32_t(GDN_FLAG_GATE_CHANNEL))) return GDN_EUNSUPPORTED;
    if (p->num_state_slots < 0 || (!state_indices && p->num_state_slots < p->num_seqs)) return GDN_EINVAL;
    if (int64_t(p->num_seqs) * p->hv > INT32_MAX - 65536) return GDN_EINVAL;
    if (p->num_seqs > 0) {
        if (!x || !state || !out || !gate_ok(p, g)) return GDN_EINVAL;
        if (!aligned16(x) || !aligned16(state) || !aligned16(out) || !aligned4(state_indices)) return GDN_EINVAL;
        if (clash({rows_of(p, out), states_of(p, state, size_t(p->num_state_slots))},
                  {rows_of(p, x), gates_of(p, g), {state_indices, size_t(p->num_seqs) * sizeof(int32_t)}}, 1, 1))
            return GDN_EINVAL;
    }
    int *status = status_ptr();
    if (!status) return GDN_ECUDA;
    return cuda_status(launch_linrec_step(x, g, state, state_indices, out, p->num_seqs, p->hv, p->num_state_slots,
                                          p->io_dtype, p->flags & GDN_FLAG_GATE_CHANNEL, status,
                                          static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace gdn {
namespace {

int check_layernorm(const gdn_problem *p) {
    if (!p || p->dv <= 0 || p->total_tokens < 0) return GDN_EINVAL;
    if (p->io_dtype != GDN_DT_F32 && p->io_dtype != GDN_DT_BF16) return GDN_EINVAL;
    if (p->total_tokens > INT32_MAX - 65536) return GDN_EINVAL;  // rows past the end stay in int
    return p->dv > kLayerNormMaxWidth ? GDN_EUNSUPPORTED : GDN_OK;
}

// the norm's tensors: rows [total_tokens, dv], one value a row, one a column
Span norm_rows(const gdn_problem *p, const void *x) { return {x, io_bytes(p, size_t(p->total_tokens) * p->dv)}; }
Span row_stats(const gdn_problem *p, const void *s) { return {s, size_t(p->total_tokens) * sizeof(float)}; }
Span columns(const gdn_problem *p, const void *w) { return {w, size_t(p->dv) * sizeof(float)}; }

bool workspace_ok(const void *ws, size_t have, size_t need) {
    return ws && !(reinterpret_cast<uintptr_t>(ws) & 255u) && have >= need;
}

}  // namespace
}  // namespace gdn

extern "C" {

int gdn_layernorm(const gdn_problem *p, const void *x, const float *weight, const float *bias, float eps, void *y,
                  float *mean, float *rstd, void *stream) {
    const int st = check_layernorm(p);
    if (st) return st;
    if (!(eps >= 0.f) || !aligned16(weight) || !aligned16(bias)) return GDN_EINVAL;
    if (p->total_tokens > 0) {
        if (!x || !y || !aligned16(x) || !aligned16(y) || !aligned4(mean) || !aligned4(rstd)) return GDN_EINVAL;
        if (clash({norm_rows(p, y), row_stats(p, mean), row_stats(p, rstd)},
                  {norm_rows(p, x), columns(p, weight), columns(p, bias)}, 1, 1))
            return GDN_EINVAL;
    }
    int *status = status_ptr();
    if (!status) return GDN_ECUDA;
    return cuda_status(launch_layernorm(x, weight, bias, eps, y, mean, rstd, p->total_tokens, p->dv, p->io_dtype,
                                        status, g_wait_ns.load(std::memory_order_relaxed),
                                        static_cast<cudaStream_t>(stream)));
}

size_t gdn_layernorm_bwd_workspace_size(const gdn_problem *p) {
    return check_layernorm(p) == GDN_OK ? layernorm_bwd_workspace(p->total_tokens, p->dv, p->io_dtype) : 0;
}

int gdn_layernorm_bwd(const gdn_problem *p, const void *dy, const void *x, const float *mean, const float *rstd,
                      const float *weight, void *dx, float *dweight, float *dbias, void *workspace,
                      size_t workspace_bytes, void *stream) {
    const int st = check_layernorm(p);
    if (st) return st;
    if (!aligned16(weight) || !aligned16(dweight) || !aligned16(dbias)) return GDN_EINVAL;
    const size_t need = dweight || dbias ? gdn_layernorm_bwd_workspace_size(p) : 0;
    // (the sums are written when all inputs have been read)
    if (clash({norm_rows(p, dx), {workspace, need}},
              {norm_rows(p, dy), norm_rows(p, x), row_stats(p, mean), row_stats(p, rstd), columns(p, weight)}, 1, 2) ||
        clash({norm_rows(p, dx), {workspace, need}, columns(p, dweight), columns(p, dbias)}, {}))
        return GDN_EINVAL;
    if (p->total_tokens > 0) {
        if (!dy || !x || !mean || !rstd || !dx) return GDN_EINVAL;
        if (!aligned16(dy) || !aligned16(x) || !aligned16(dx) || !aligned4(mean) || !aligned4(rstd))
            return GDN_EINVAL;
        if ((dweight || dbias) && !workspace_ok(workspace, workspace_bytes, need))
            return GDN_EINVAL;
    }
    int *status = status_ptr();
    if (!status) return GDN_ECUDA;
    return cuda_status(launch_layernorm_bwd(dy, x, mean, rstd, weight, dx, dweight, dbias, workspace, p->total_tokens,
                                            p->dv, p->io_dtype, status, g_wait_ns.load(std::memory_order_relaxed),
                                            static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace gdn {
namespace {

int check_gate_norm(const gdn_problem *p) {
    if (!p || p->hv <= 0 || p->total_tokens < 0) return GDN_EINVAL;
    if (p->io_dtype != GDN_DT_F32 && p->io_dtype != GDN_DT_BF16) return GDN_EINVAL;
    if (p->dv != kHeadDim) return p->dv > 0 ? GDN_EUNSUPPORTED : GDN_EINVAL;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

extern "C" {

size_t gdn_gated_rmsnorm_bwd_workspace_size(const gdn_problem *p) {
    if (check_gate_norm(p) != GDN_OK) return 0;
    return gated_rmsnorm_bwd_workspace((long long)p->total_tokens * p->hv, p->io_dtype);
}

int gdn_gated_rmsnorm_bwd(const gdn_problem *p, const void *dy, const void *o, const void *z, const float *weight,
                          float eps, void *d_o, void *d_z, float *d_weight, void *workspace, size_t workspace_bytes,
                          void *stream) {
    const int st = check_gate_norm(p);
    if (st) return st;
    if (!(eps >= 0.f) || !aligned16(d_weight)) return GDN_EINVAL;
    const long long rows = (long long)p->total_tokens * p->hv;
    if (rows > 0) {
        if (!dy || !o || !z || !weight || !d_o || !d_z) return GDN_EINVAL;
        if (!aligned16(dy) || !aligned16(o) || !aligned16(z) || !aligned16(weight) || !aligned16(d_o) ||
            !aligned16(d_z))
            return GDN_EINVAL;
        const size_t need = d_weight ? gdn_gated_rmsnorm_bwd_workspace_size(p) : 0;
        if (d_weight && !workspace_ok(workspace, workspace_bytes, need)) return GDN_EINVAL;
        const size_t columns = kHeadDim * sizeof(float);
        if (clash({rows_of(p, d_o), rows_of(p, d_z), {workspace, need}},
                  {rows_of(p, dy), rows_of(p, o), rows_of(p, z), {weight, columns}}, 2, 3) ||
            clash({rows_of(p, d_o), rows_of(p, d_z), {workspace, need}, {d_weight, columns}}, {}))
            return GDN_EINVAL;
    }
    return cuda_status(launch_gated_rmsnorm_bwd(dy, o, z, weight, eps, d_o, d_z, d_weight, workspace, rows,
                                                p->io_dtype, static_cast<cudaStream_t>(stream)));
}

int gdn_read_device_status(void *stream, int clear) {
    int *status = status_ptr();
    if (!status) return GDN_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int host = 0;
    if (cudaMemcpyAsync(&host, status, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess) return GDN_ECUDA;
    if (clear && cudaMemsetAsync(status, 0, sizeof(int), s) != cudaSuccess) return GDN_ECUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return GDN_ECUDA;
    return host;
}

int gdn_get_device_status(void *stream) { return gdn_read_device_status(stream, 1); }

int gdn_set_wait_limit_ns(unsigned long long ns) {
    g_wait_ns.store(ns ? ns : kDefaultWaitNs, std::memory_order_relaxed);
    return GDN_OK;
}

}  // extern "C"
