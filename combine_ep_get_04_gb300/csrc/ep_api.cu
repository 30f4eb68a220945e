// ep_api.cu -- the C ABI declared in include/ep.h: host-side argument checks,
// launch-shape choice and error reporting.  Every step of the work runs in
// the kernels of layout.cu, dispatch.cu and combine.cu on the caller's stream.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "ep.h"
#include "block_kernels.h"

namespace {

thread_local std::string g_last_error;

ep_status_t fail(ep_status_t st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return st;
}

ep_status_t ok() { return EP_OK; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Checks the shape; returns EP_OK or a failure with the reason recorded.
ep_status_t check_shape(const ep_shape_t* s) {
    if (s == nullptr) return fail(EP_ERR_INVALID_ARG, "shape is NULL");
    if (s->T < 0) return fail(EP_ERR_INVALID_ARG, "T = %d < 0", s->T);
    if (s->H <= 0 || s->H % 8 != 0) return fail(EP_ERR_INVALID_ARG, "H = %d must be a positive multiple of 8", s->H);
    if (s->E < 1) return fail(EP_ERR_INVALID_ARG, "E = %d < 1", s->E);
    if (s->E > EP_MAX_EXPERTS) return fail(EP_ERR_UNSUPPORTED, "E = %d > %d", s->E, EP_MAX_EXPERTS);
    if (s->k < 1 || s->k > s->E) return fail(EP_ERR_INVALID_ARG, "k = %d must be in [1, E = %d]", s->k, s->E);
    if (s->k > EP_MAX_TOPK) return fail(EP_ERR_UNSUPPORTED, "k = %d > %d", s->k, EP_MAX_TOPK);
    if (s->num_partitions < 1 || s->E % s->num_partitions != 0)
        return fail(EP_ERR_INVALID_ARG, "num_partitions = %d must divide E = %d", s->num_partitions, s->E);
    if (s->mode != EP_LAYOUT_PACKED && s->mode != EP_LAYOUT_CAPACITY)
        return fail(EP_ERR_INVALID_ARG, "mode = %d is not a layout mode", s->mode);
    if (s->mode == EP_LAYOUT_CAPACITY && s->capacity < 1)
        return fail(EP_ERR_INVALID_ARG, "capacity = %d < 1 in capacity mode", s->capacity);
    const int64_t N = (int64_t)s->T * s->k;
    const int64_t R = s->mode == EP_LAYOUT_PACKED ? N : (int64_t)s->E * s->capacity;
    if (N > INT32_MAX || R > INT32_MAX)
        return fail(EP_ERR_UNSUPPORTED, "T*k = %lld or R = %lld exceeds 2^31-1", (long long)N, (long long)R);
    return ok();
}

int64_t rows_of(const ep_shape_t* s) {
    return s->mode == EP_LAYOUT_PACKED ? (int64_t)s->T * s->k : (int64_t)s->E * s->capacity;
}

// The current device must be an sm_103 part (the only code this library holds).
// What a device is does not change, so each is asked once.
ep_status_t device_info(int* num_sms) {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> known[kMaxDevices];     // SMs of an sm_103 device, 0: not asked yet
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail(EP_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    if (dev >= 0 && dev < kMaxDevices && (*num_sms = known[dev].load(std::memory_order_relaxed)) > 0) return ok();
    int major = 0, minor = 0;
    e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return fail(EP_ERR_CUDA, "cudaDeviceGetAttribute: %s", cudaGetErrorString(e));
    if (major != 10 || minor != 3)
        return fail(EP_ERR_UNSUPPORTED, "device %d is sm_%d%d; this library holds sm_103a code only", dev, major,
                    minor);
    if (dev >= 0 && dev < kMaxDevices) known[dev].store(*num_sms, std::memory_order_relaxed);
    return ok();
}

ep_status_t launched(cudaError_t e, const char* what) {
    if (e != cudaSuccess) return fail(EP_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return ok();
}

// ------------------------------------------------------------------ route

ep_status_t check_route(const ep_route_t* r) {
    if (r == nullptr) return fail(EP_ERR_INVALID_ARG, "route is NULL");
    if (r->T < 0) return fail(EP_ERR_INVALID_ARG, "T = %d < 0", r->T);
    if (r->E < 1) return fail(EP_ERR_INVALID_ARG, "E = %d < 1", r->E);
    if (r->E > EP_MAX_EXPERTS) return fail(EP_ERR_UNSUPPORTED, "E = %d > %d", r->E, EP_MAX_EXPERTS);
    if (r->k < 1 || r->k > r->E) return fail(EP_ERR_INVALID_ARG, "k = %d must be in [1, E = %d]", r->k, r->E);
    if (r->k > EP_MAX_TOPK) return fail(EP_ERR_UNSUPPORTED, "k = %d > %d", r->k, EP_MAX_TOPK);
    if (r->groups < 1 || r->E % r->groups != 0)
        return fail(EP_ERR_INVALID_ARG, "groups = %d must divide E = %d", r->groups, r->E);
    if (r->groups > EP_MAX_ROUTE_GROUPS)
        return fail(EP_ERR_UNSUPPORTED, "groups = %d > %d", r->groups, EP_MAX_ROUTE_GROUPS);
    if (r->topk_groups < 1 || r->topk_groups > r->groups)
        return fail(EP_ERR_INVALID_ARG, "topk_groups = %d must be in [1, groups = %d]", r->topk_groups, r->groups);
    if (r->full_softmax != 0 && r->full_softmax != 1)
        return fail(EP_ERR_INVALID_ARG, "full_softmax = %d must be 0 or 1", r->full_softmax);
    if (r->logits_type != EP_TYPE_BF16 && r->logits_type != EP_TYPE_F32)
        return fail(EP_ERR_INVALID_ARG, "logits_type = %d is not a type", r->logits_type);
    if (r->num_seqs < 1) return fail(EP_ERR_INVALID_ARG, "num_seqs = %d < 1", r->num_seqs);
    if (r->num_seqs > 65535) return fail(EP_ERR_UNSUPPORTED, "num_seqs = %d > 65535", r->num_seqs);
    if ((int64_t)r->T * r->k > INT32_MAX)
        return fail(EP_ERR_UNSUPPORTED, "T*k = %lld exceeds 2^31-1", (long long)r->T * r->k);
    return ok();
}

ep::RouteParams route_params(const ep_route_t* r) {
    ep::RouteParams p{};
    p.T = r->T;
    p.E = r->E;
    p.k = r->k;
    p.groups = r->groups;
    p.topk_groups = r->topk_groups;
    p.full_softmax = r->full_softmax;
    p.f32 = r->logits_type == EP_TYPE_F32 ? 1 : 0;
    p.S = r->num_seqs;
    p.balance_coef = r->balance_coef;
    p.z_coef = r->z_coef;
    return p;
}

ep_status_t check_logits(const ep_route_t* r, const void* logits, int64_t ld) {
    const uintptr_t mask = r->logits_type == EP_TYPE_F32 ? 3u : 1u;
    if (logits == nullptr) return fail(EP_ERR_INVALID_ARG, "logits is NULL");
    if (reinterpret_cast<uintptr_t>(logits) & mask) return fail(EP_ERR_INVALID_ARG, "logits is not aligned to its elements");
    if (ld < r->E) return fail(EP_ERR_INVALID_ARG, "ld = %lld < E = %d", (long long)ld, r->E);
    return ok();
}

// -------------------------------------------------------------- expert w4

ep_status_t check_w4(const ep_w4_t* w) {
    if (w == nullptr) return fail(EP_ERR_INVALID_ARG, "w is NULL");
    if (w->E < 1) return fail(EP_ERR_INVALID_ARG, "E = %d < 1", w->E);
    if (w->E > EP_MAX_EXPERTS) return fail(EP_ERR_UNSUPPORTED, "E = %d > %d", w->E, EP_MAX_EXPERTS);
    if (w->N <= 0 || w->N % 8 != 0) return fail(EP_ERR_INVALID_ARG, "N = %d must be a positive multiple of 8", w->N);
    if (w->K <= 0 || w->K % 8 != 0) return fail(EP_ERR_INVALID_ARG, "K = %d must be a positive multiple of 8", w->K);
    if (w->group != 32 && w->group != 64 && w->group != 128)
        return fail(EP_ERR_INVALID_ARG, "group = %d must be 32, 64 or 128", w->group);
    if (w->paired != 0 && w->paired != 1) return fail(EP_ERR_INVALID_ARG, "paired = %d must be 0 or 1", w->paired);
    if (w->N > 1 << 24 || w->K > 1 << 24 || !ep::w4_packs({w->E, w->N, w->K, w->group, w->paired}))
        return fail(EP_ERR_UNSUPPORTED, "weights [%d, %d, %d] are too large", w->E, w->N, w->K);
    return ok();
}

// ------------------------------------------------------------- block norm

ep_status_t check_norm(const ep_norm_t* s) {
    if (s == nullptr) return fail(EP_ERR_INVALID_ARG, "norm is NULL");
    if (s->T < 0) return fail(EP_ERR_INVALID_ARG, "T = %d < 0", s->T);
    if (s->H <= 0 || s->H % 8 != 0) return fail(EP_ERR_INVALID_ARG, "H = %d must be a positive multiple of 8", s->H);
    if (s->H > EP_MAX_NORM_WIDTH) return fail(EP_ERR_UNSUPPORTED, "H = %d > %d", s->H, EP_MAX_NORM_WIDTH);
    if (s->stream_type != EP_TYPE_BF16 && s->stream_type != EP_TYPE_F32)
        return fail(EP_ERR_INVALID_ARG, "stream_type = %d is not a type", s->stream_type);
    if (s->gate_kind != EP_GATE_NONE && s->gate_kind != EP_GATE_CHANNEL && s->gate_kind != EP_GATE_TOKEN)
        return fail(EP_ERR_INVALID_ARG, "gate_kind = %d is not a gate kind", s->gate_kind);
    // the backward pass multiplies two reciprocal roots, each up to eps^-1/2
    if (!(s->eps >= 1e-30f) || !(s->eps <= 1e30f)) return fail(EP_ERR_INVALID_ARG, "eps = %g must be in [1e-30, 1e30]", (double)s->eps);
    return ok();
}

// What both directions take in.
ep_status_t check_norm_inputs(const ep_norm_t* s, const void* h, int64_t ld_h, const void* y, int64_t ld_y,
                              const float* w_post, const float* gate, const float* w_pre) {
    if (h == nullptr) return fail(EP_ERR_INVALID_ARG, "h is NULL");
    if (ld_h < s->H || ld_h % 8 != 0) return fail(EP_ERR_INVALID_ARG, "ld_h = %lld must be a multiple of 8 and at least H = %d", (long long)ld_h, s->H);
    if (y != nullptr && (ld_y < s->H || ld_y % 8 != 0))
        return fail(EP_ERR_INVALID_ARG, "ld_y = %lld must be a multiple of 8 and at least H = %d", (long long)ld_y, s->H);
    if (y == nullptr && (w_post != nullptr || s->gate_kind != EP_GATE_NONE))
        return fail(EP_ERR_INVALID_ARG, "w_post and gate need y");
    if ((gate != nullptr) != (s->gate_kind != EP_GATE_NONE))
        return fail(EP_ERR_INVALID_ARG, "gate and gate_kind = %d do not agree", s->gate_kind);
    if (!aligned16(h) || !aligned16(y) || !aligned16(w_post) || !aligned16(w_pre) ||
        (s->gate_kind == EP_GATE_CHANNEL && !aligned16(gate)))
        return fail(EP_ERR_INVALID_ARG, "h, y, w_post, w_pre and a channel gate must be 16-byte aligned");
    return ok();
}

// ------------------------------------------------- dropout and layer norm

// Sets *d; EP_OK, or the reason why p is no probability.
ep_status_t set_dropout(ep::Dropout* d, double p, const int64_t* rng, uint64_t site) {
    if (!(p >= 0.0 && p <= 1.0)) return fail(EP_ERR_INVALID_ARG, "p = %g must be in [0, 1]", p);
    if (reinterpret_cast<uintptr_t>(rng) & 7u) return fail(EP_ERR_INVALID_ARG, "rng must be 8-byte aligned");
    *d = ep::Dropout{};
    const uint64_t limit = (uint64_t)nearbyint(p * 65536.0);
    d->rng = limit != 0 ? rng : nullptr;
    d->site = site;
    d->most = (uint32_t)((limit << 16) - 1);
    d->scale = limit < 65536 ? (float)(65536.0 / (65536.0 - (double)limit)) : 0.f;
    return ok();
}

ep_status_t check_layer_norm(const ep_layer_norm_t* s) {
    if (s == nullptr) return fail(EP_ERR_INVALID_ARG, "norm is NULL");
    if (s->T < 0) return fail(EP_ERR_INVALID_ARG, "T = %d < 0", s->T);
    if (s->H <= 0 || s->H % 8 != 0) return fail(EP_ERR_INVALID_ARG, "H = %d must be a positive multiple of 8", s->H);
    if (s->H > EP_MAX_NORM_WIDTH) return fail(EP_ERR_UNSUPPORTED, "H = %d > %d", s->H, EP_MAX_NORM_WIDTH);
    if (s->stream_type != EP_TYPE_BF16 && s->stream_type != EP_TYPE_F32)
        return fail(EP_ERR_INVALID_ARG, "stream_type = %d is not a type", s->stream_type);
    if (!(s->eps >= 1e-30f) || !(s->eps <= 1e30f)) return fail(EP_ERR_INVALID_ARG, "eps = %g must be in [1e-30, 1e30]", (double)s->eps);
    ep::Dropout d;
    return set_dropout(&d, s->p, nullptr, s->site);
}

ep_status_t check_norm_rows(const char* name, const void* rows, int64_t ld, int H) {
    if (ld < H || ld % 8 != 0) return fail(EP_ERR_INVALID_ARG, "ld_%s = %lld must be a multiple of 8 and at least H = %d", name, (long long)ld, H);
    if (!aligned16(rows)) return fail(EP_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
    return ok();
}

// ---------------------------------------------------------- 8-bit integers

ep_status_t check_i8(const ep_i8_t* w) {
    if (w == nullptr) return fail(EP_ERR_INVALID_ARG, "w is NULL");
    if (w->E < 1) return fail(EP_ERR_INVALID_ARG, "E = %d < 1", w->E);
    if (w->E > EP_MAX_EXPERTS) return fail(EP_ERR_UNSUPPORTED, "E = %d > %d", w->E, EP_MAX_EXPERTS);
    if (w->N <= 0 || w->N % 8 != 0) return fail(EP_ERR_INVALID_ARG, "N = %d must be a positive multiple of 8", w->N);
    if (w->K <= 0 || w->K % 16 != 0) return fail(EP_ERR_INVALID_ARG, "K = %d must be a positive multiple of 16", w->K);
    if (w->paired != 0 && w->paired != 1) return fail(EP_ERR_INVALID_ARG, "paired = %d must be 0 or 1", w->paired);
    if (w->N > 1 << 24 || w->K > 1 << 24 || !ep::i8_packs({w->E, w->N, w->K, w->paired}))
        return fail(EP_ERR_UNSUPPORTED, "weights [%d, %d, %d] are too large", w->E, w->N, w->K);
    return ok();
}

// Which rows hold a copy.
ep_status_t check_rows(int E, int32_t mode, int32_t capacity, int64_t R, const int32_t* counts, const int32_t* offsets, bool all_rows) {
    if (mode != EP_LAYOUT_PACKED && mode != EP_LAYOUT_CAPACITY)
        return fail(EP_ERR_INVALID_ARG, "mode = %d is not a layout mode", mode);
    if (R < 0) return fail(EP_ERR_INVALID_ARG, "R must not be negative");
    if (R > INT32_MAX) return fail(EP_ERR_UNSUPPORTED, "R = %lld exceeds 2^31-1", (long long)R);
    if (mode == EP_LAYOUT_CAPACITY && (capacity < 1 || R < (int64_t)E * capacity))
        return fail(EP_ERR_INVALID_ARG, "capacity = %d needs at least 1 and R >= E*capacity", capacity);
    if (R > 0 && (mode == EP_LAYOUT_CAPACITY ? counts == nullptr : offsets == nullptr && !all_rows))
        return fail(EP_ERR_INVALID_ARG, "counts (capacity mode) / offsets (packed) is NULL");
    return ok();
}

}  // namespace

namespace ep {
void record_last_error(const char* msg) { g_last_error = msg; }
}  // namespace ep

extern "C" {

int32_t ep_abi_version(void) { return 101; }

const char* ep_status_string(ep_status_t st) {
    switch (st) {
        case EP_OK: return "ok";
        case EP_ERR_INVALID_ARG: return "invalid argument";
        case EP_ERR_UNSUPPORTED: return "unsupported";
        case EP_ERR_CUDA: return "CUDA error";
    }
    return "unknown status";
}

const char* ep_status_str(ep_status_t st) { return ep_status_string(st); }

const char* ep_last_error(void) { return g_last_error.c_str(); }

int64_t ep_recv_rows(const ep_shape_t* shape) {
    if (check_shape(shape) != EP_OK) return -1;
    return rows_of(shape);
}

size_t ep_layout_workspace_bytes(const ep_shape_t* shape) {
    if (check_shape(shape) != EP_OK) return (size_t)-1;
    return ep::layout_workspace_bytes((int64_t)shape->T * shape->k, shape->E);
}

ep_status_t ep_get_layout(const ep_shape_t* shape, const int32_t* topk_idx, int32_t* counts, int32_t* offsets,
                          int32_t* part_counts, int32_t* part_offsets, int32_t* slot_of, int32_t* src_token,
                          int32_t* src_k, void* workspace, size_t workspace_bytes, uint32_t* err_flags,
                          ep_stream_t stream) {
    ep_status_t st = check_shape(shape);
    if (st != EP_OK) return st;
    const int64_t N = (int64_t)shape->T * shape->k;
    const int64_t R = rows_of(shape);
    if (N > 0 && (topk_idx == nullptr || slot_of == nullptr))
        return fail(EP_ERR_INVALID_ARG, "topk_idx / slot_of is NULL");
    if (counts == nullptr || offsets == nullptr || part_counts == nullptr || part_offsets == nullptr)
        return fail(EP_ERR_INVALID_ARG, "counts / offsets / part_counts / part_offsets is NULL");
    if (R > 0 && (src_token == nullptr || src_k == nullptr))
        return fail(EP_ERR_INVALID_ARG, "src_token / src_k is NULL");
    const size_t need = ep::layout_workspace_bytes(N, shape->E);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
        return fail(EP_ERR_INVALID_ARG, "workspace of %zu bytes given, %zu needed", workspace_bytes, need);
    if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 3u))
        return fail(EP_ERR_INVALID_ARG, "workspace is not 4-byte aligned");
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;

    ep::LayoutParams p{};
    p.topk_idx = topk_idx;
    p.counts = counts;
    p.offsets = offsets;
    p.part_counts = part_counts;
    p.part_offsets = part_offsets;
    p.slot_of = slot_of;
    p.src_token = src_token;
    p.src_k = src_k;
    p.hist = need > 0 ? static_cast<int32_t*>(workspace) : nullptr;
    p.err_flags = err_flags;
    p.N = N;
    p.R = R;
    p.E = shape->E;
    p.P = shape->num_partitions;
    p.k = shape->k;
    p.mode = shape->mode;
    p.cap = shape->capacity;
    return launched(ep::launch_layout(p, num_sms, reinterpret_cast<cudaStream_t>(stream)), "layout launch");
}

ep_status_t ep_dispatch(const ep_shape_t* shape, const void* x, const float* topk_w, const int32_t* slot_of,
                        int32_t payload, void* recv, void* recv_scales, float* recv_w, uint32_t* err_flags,
                        ep_stream_t stream) {
    ep_status_t st = check_shape(shape);
    if (st != EP_OK) return st;
    if (payload != EP_PAYLOAD_BF16 && payload != EP_PAYLOAD_FP8_E4M3 && payload != EP_PAYLOAD_FP8_E4M3_UE8M0)
        return fail(EP_ERR_INVALID_ARG, "payload = %d is not a payload format", payload);
    const bool fp8 = payload != EP_PAYLOAD_BF16;
    const bool ue8m0 = payload == EP_PAYLOAD_FP8_E4M3_UE8M0;
    if (fp8 && shape->H % 128 != 0) return fail(EP_ERR_INVALID_ARG, "fp8 payload needs H %% 128 == 0 (H = %d)", shape->H);
    if (shape->T == 0) return ok();
    if (x == nullptr || slot_of == nullptr || recv == nullptr)
        return fail(EP_ERR_INVALID_ARG, "x / slot_of / recv is NULL");
    if (!aligned16(x) || !aligned16(recv)) return fail(EP_ERR_INVALID_ARG, "x and recv must be 16-byte aligned");
    if (fp8 && (recv_scales == nullptr || (!ue8m0 && !aligned16(recv_scales))))
        return fail(EP_ERR_INVALID_ARG, "fp8 payload needs recv_scales (16-byte aligned for f32 scales)");
    if (recv_w != nullptr && topk_w == nullptr) return fail(EP_ERR_INVALID_ARG, "recv_w needs topk_w");
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;

    ep::DispatchParams p{};
    p.x = x;
    p.topk_w = topk_w;
    p.slot_of = slot_of;
    p.recv = recv;
    p.recv_scales = recv_scales;
    p.ue8m0 = ue8m0 ? 1 : 0;
    p.recv_w = recv_w;
    p.err_flags = err_flags;
    p.R = rows_of(shape);
    p.T = shape->T;
    p.H = shape->H;
    p.k = shape->k;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return launched(fp8 ? ep::launch_dispatch_fp8(p, num_sms, s) : ep::launch_dispatch_bf16(p, num_sms, s),
                    "dispatch launch");
}

ep_status_t ep_layout_dispatch(const ep_shape_t* shape, const int32_t* topk_idx, const void* x,
                               const float* topk_w, int32_t payload, int32_t* counts, int32_t* offsets,
                               int32_t* part_counts, int32_t* part_offsets, int32_t* slot_of, int32_t* src_token,
                               int32_t* src_k, void* recv, void* recv_scales, float* recv_w, void* workspace,
                               size_t workspace_bytes, uint32_t* err_flags, ep_stream_t stream) {
    ep_status_t st = check_shape(shape);
    if (st != EP_OK) return st;
    const int64_t N = (int64_t)shape->T * shape->k;
    if (!ep::fused_layout_dispatch_fits(N, shape->T, shape->E) || shape->T == 0) {
        st = ep_get_layout(shape, topk_idx, counts, offsets, part_counts, part_offsets, slot_of, src_token, src_k,
                           workspace, workspace_bytes, err_flags, stream);
        if (st != EP_OK) return st;
        return ep_dispatch(shape, x, topk_w, slot_of, payload, recv, recv_scales, recv_w, err_flags, stream);
    }
    // The same checks as ep_get_layout and ep_dispatch, before anything is launched.
    if (payload != EP_PAYLOAD_BF16 && payload != EP_PAYLOAD_FP8_E4M3 && payload != EP_PAYLOAD_FP8_E4M3_UE8M0)
        return fail(EP_ERR_INVALID_ARG, "payload = %d is not a payload format", payload);
    const bool fp8 = payload != EP_PAYLOAD_BF16;
    const bool ue8m0 = payload == EP_PAYLOAD_FP8_E4M3_UE8M0;
    if (fp8 && shape->H % 128 != 0) return fail(EP_ERR_INVALID_ARG, "fp8 payload needs H %% 128 == 0 (H = %d)", shape->H);
    if (topk_idx == nullptr || slot_of == nullptr || x == nullptr || recv == nullptr)
        return fail(EP_ERR_INVALID_ARG, "topk_idx / slot_of / x / recv is NULL");
    if (counts == nullptr || offsets == nullptr || part_counts == nullptr || part_offsets == nullptr ||
        src_token == nullptr || src_k == nullptr)
        return fail(EP_ERR_INVALID_ARG, "counts / offsets / part_counts / part_offsets / src_token / src_k is NULL");
    if (!aligned16(x) || !aligned16(recv)) return fail(EP_ERR_INVALID_ARG, "x and recv must be 16-byte aligned");
    if (fp8 && (recv_scales == nullptr || (!ue8m0 && !aligned16(recv_scales))))
        return fail(EP_ERR_INVALID_ARG, "fp8 payload needs recv_scales (16-byte aligned for f32 scales)");
    if (recv_w != nullptr && topk_w == nullptr) return fail(EP_ERR_INVALID_ARG, "recv_w needs topk_w");
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;

    ep::FusedLaunch f{};
    f.topk_idx = topk_idx;
    f.x = x;
    f.topk_w = topk_w;
    f.counts = counts;
    f.offsets = offsets;
    f.part_counts = part_counts;
    f.part_offsets = part_offsets;
    f.slot_of = slot_of;
    f.src_token = src_token;
    f.src_k = src_k;
    f.recv = recv;
    f.recv_scales = recv_scales;
    f.recv_w = recv_w;
    f.err_flags = err_flags;
    f.R = rows_of(shape);
    f.T = shape->T;
    f.H = shape->H;
    f.E = shape->E;
    f.k = shape->k;
    f.P = shape->num_partitions;
    f.mode = shape->mode;
    f.cap = shape->capacity;
    f.fp8 = fp8 ? 1 : 0;
    f.ue8m0 = ue8m0 ? 1 : 0;
    return launched(ep::launch_layout_dispatch(f, num_sms, reinterpret_cast<cudaStream_t>(stream)),
                    "layout+dispatch launch");
}

ep_status_t ep_combine(const ep_shape_t* shape, const void* y, const float* topk_w, const int32_t* slot_of,
                       void* out, uint32_t* err_flags, ep_stream_t stream) {
    ep_status_t st = check_shape(shape);
    if (st != EP_OK) return st;
    if (shape->T == 0) return ok();
    if (y == nullptr || slot_of == nullptr || out == nullptr)
        return fail(EP_ERR_INVALID_ARG, "y / slot_of / out is NULL");
    if (!aligned16(y) || !aligned16(out)) return fail(EP_ERR_INVALID_ARG, "y and out must be 16-byte aligned");
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;

    ep::CombineParams p{};
    p.y = y;
    p.topk_w = topk_w;
    p.slot_of = slot_of;
    p.out = out;
    p.err_flags = err_flags;
    p.R = rows_of(shape);
    p.T = shape->T;
    p.H = shape->H;
    p.k = shape->k;
    return launched(ep::launch_combine(p, num_sms, reinterpret_cast<cudaStream_t>(stream)), "combine launch");
}

ep_status_t ep_combine_fp8(const ep_shape_t* shape, const void* y, const void* y_scales, int32_t payload,
                           const float* topk_w, const int32_t* slot_of, void* out, uint32_t* err_flags,
                           ep_stream_t stream) {
    ep_status_t st = check_shape(shape);
    if (st != EP_OK) return st;
    if (payload != EP_PAYLOAD_FP8_E4M3 && payload != EP_PAYLOAD_FP8_E4M3_UE8M0)
        return fail(EP_ERR_INVALID_ARG, "payload = %d is not an fp8 payload format", payload);
    if (shape->H % 128 != 0) return fail(EP_ERR_INVALID_ARG, "fp8 expert outputs need H %% 128 == 0 (H = %d)", shape->H);
    if (shape->T == 0) return ok();
    const bool ue8m0 = payload == EP_PAYLOAD_FP8_E4M3_UE8M0;
    if (y == nullptr || y_scales == nullptr || slot_of == nullptr || out == nullptr)
        return fail(EP_ERR_INVALID_ARG, "y / y_scales / slot_of / out is NULL");
    if (!aligned16(y) || !aligned16(out)) return fail(EP_ERR_INVALID_ARG, "y and out must be 16-byte aligned");
    if (!ue8m0 && (reinterpret_cast<uintptr_t>(y_scales) & 3u))
        return fail(EP_ERR_INVALID_ARG, "f32 y_scales must be 4-byte aligned");
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;

    ep::CombineParams p{};
    p.y = y;
    p.y_scales = y_scales;
    p.fp8 = 1;
    p.ue8m0 = ue8m0 ? 1 : 0;
    p.topk_w = topk_w;
    p.slot_of = slot_of;
    p.out = out;
    p.err_flags = err_flags;
    p.R = rows_of(shape);
    p.T = shape->T;
    p.H = shape->H;
    p.k = shape->k;
    return launched(ep::launch_combine(p, num_sms, reinterpret_cast<cudaStream_t>(stream)), "combine launch");
}

size_t ep_combine_src_workspace_bytes(const ep_shape_t* shape) {
    if (check_shape(shape) != EP_OK) return 0;
    return ep::combine_src_workspace_bytes(shape->T, shape->k);
}

ep_status_t ep_combine_src(const ep_shape_t* shape, const void* y, const void* y_scales, int32_t payload,
                           const float* row_w, const int32_t* src_token, const int32_t* src_k, void* out,
                           void* workspace, size_t workspace_bytes, uint32_t* err_flags, ep_stream_t stream) {
    ep_status_t st = check_shape(shape);
    if (st != EP_OK) return st;
    if (payload != EP_PAYLOAD_BF16 && payload != EP_PAYLOAD_FP8_E4M3 && payload != EP_PAYLOAD_FP8_E4M3_UE8M0)
        return fail(EP_ERR_INVALID_ARG, "payload = %d is not a payload format", payload);
    const bool fp8 = payload != EP_PAYLOAD_BF16;
    const bool ue8m0 = payload == EP_PAYLOAD_FP8_E4M3_UE8M0;
    if (fp8 && shape->H % 128 != 0)
        return fail(EP_ERR_INVALID_ARG, "fp8 expert outputs need H %% 128 == 0 (H = %d)", shape->H);
    if (shape->T == 0) return ok();
    if (y == nullptr || out == nullptr || workspace == nullptr)
        return fail(EP_ERR_INVALID_ARG, "y / out / workspace is NULL");
    const int64_t R = rows_of(shape);
    if (R > 0 && (src_token == nullptr || src_k == nullptr))
        return fail(EP_ERR_INVALID_ARG, "src_token / src_k is NULL");
    if (fp8 && y_scales == nullptr) return fail(EP_ERR_INVALID_ARG, "fp8 expert outputs need y_scales");
    if (!aligned16(y) || !aligned16(out)) return fail(EP_ERR_INVALID_ARG, "y and out must be 16-byte aligned");
    if (fp8 && !ue8m0 && (reinterpret_cast<uintptr_t>(y_scales) & 3u))
        return fail(EP_ERR_INVALID_ARG, "f32 y_scales must be 4-byte aligned");
    const size_t need = ep::combine_src_workspace_bytes(shape->T, shape->k);
    if (workspace_bytes < need)
        return fail(EP_ERR_INVALID_ARG, "workspace of %zu bytes given, %zu needed", workspace_bytes, need);
    if (reinterpret_cast<uintptr_t>(workspace) & 3u) return fail(EP_ERR_INVALID_ARG, "workspace is not 4-byte aligned");
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;

    ep::CombineSrcParams p{};
    p.base.y = y;
    p.base.y_scales = fp8 ? y_scales : nullptr;
    p.base.fp8 = fp8 ? 1 : 0;
    p.base.ue8m0 = ue8m0 ? 1 : 0;
    p.base.out = out;
    p.base.err_flags = err_flags;
    p.base.R = R;
    p.base.T = shape->T;
    p.base.H = shape->H;
    p.base.k = shape->k;
    p.row_w = row_w;
    p.src_token = src_token;
    p.src_k = src_k;
    p.workspace = workspace;
    return launched(ep::launch_combine_src(p, num_sms, reinterpret_cast<cudaStream_t>(stream)), "combine_src launch");
}

size_t ep_route_workspace_bytes(const ep_route_t* route) {
    if (check_route(route) != EP_OK) return (size_t)-1;
    ep::RouteParams p = route_params(route);
    return ep::route_workspace(&p, nullptr);
}

ep_status_t ep_route(const ep_route_t* route, const void* logits, int64_t ld, const float* select_bias,
                     const uint8_t* token_mask, const int32_t* seq_offsets, int32_t* topk_idx, float* topk_w,
                     float* lse, int32_t* counts, float* prob_sums, int32_t* seq_tokens, float* losses,
                     void* workspace, size_t workspace_bytes, uint32_t* err_flags, ep_stream_t stream) {
    ep_status_t st = check_route(route);
    if (st != EP_OK) return st;
    const bool sums = losses != nullptr;
    if (route->T > 0) {
        st = check_logits(route, logits, ld);
        if (st != EP_OK) return st;
        if (topk_idx == nullptr || topk_w == nullptr) return fail(EP_ERR_INVALID_ARG, "topk_idx / topk_w is NULL");
    } else if (!sums) {
        return ok();
    }
    if ((counts != nullptr) != sums || (prob_sums != nullptr) != sums || (seq_tokens != nullptr) != sums)
        return fail(EP_ERR_INVALID_ARG, "counts, prob_sums, seq_tokens and losses go together");
    ep::RouteParams p = route_params(route);
    if (sums) {
        if (lse == nullptr && route->T > 0) return fail(EP_ERR_INVALID_ARG, "the losses need lse");
        if (seq_offsets == nullptr && route->num_seqs != 1)
            return fail(EP_ERR_INVALID_ARG, "num_seqs = %d needs seq_offsets", route->num_seqs);
        const size_t need = ep::route_workspace(&p, nullptr);
        if (workspace == nullptr || workspace_bytes < need)
            return fail(EP_ERR_INVALID_ARG, "workspace of %zu bytes given, %zu needed", workspace_bytes, need);
        if (!aligned16(workspace)) return fail(EP_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
        ep::route_workspace(&p, workspace);
    }
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;
    p.logits = logits;
    p.ld = ld;
    p.select_bias = select_bias;
    p.token_mask = token_mask;
    p.seq_offsets = seq_offsets;
    p.topk_idx = topk_idx;
    p.topk_w = topk_w;
    p.lse = lse;
    p.counts = counts;
    p.prob_sums = prob_sums;
    p.seq_tokens = seq_tokens;
    p.losses = losses;
    p.err_flags = err_flags;
    return launched(ep::launch_route(p, num_sms, reinterpret_cast<cudaStream_t>(stream)), "route launch");
}

ep_status_t ep_route_backward(const ep_route_t* route, const void* logits, int64_t ld, const int32_t* seq_offsets,
                              const int32_t* topk_idx, const float* topk_w, const float* lse, const int32_t* counts,
                              const int32_t* seq_tokens, const float* d_topk_w, const float* d_losses,
                              void* d_logits, ep_stream_t stream) {
    ep_status_t st = check_route(route);
    if (st != EP_OK) return st;
    if (route->T == 0) return ok();
    st = check_logits(route, logits, ld);
    if (st != EP_OK) return st;
    if (topk_idx == nullptr || topk_w == nullptr || lse == nullptr || counts == nullptr || seq_tokens == nullptr ||
        d_logits == nullptr)
        return fail(EP_ERR_INVALID_ARG, "topk_idx / topk_w / lse / counts / seq_tokens / d_logits is NULL");
    if (reinterpret_cast<uintptr_t>(d_logits) & (route->logits_type == EP_TYPE_F32 ? 3u : 1u))
        return fail(EP_ERR_INVALID_ARG, "d_logits is not aligned to its elements");
    if (seq_offsets == nullptr && route->num_seqs != 1)
        return fail(EP_ERR_INVALID_ARG, "num_seqs = %d needs seq_offsets", route->num_seqs);
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;
    ep::RouteParams p = route_params(route);
    p.logits = logits;
    p.ld = ld;
    p.seq_offsets = seq_offsets;
    p.topk_idx = const_cast<int32_t*>(topk_idx);
    p.topk_w = const_cast<float*>(topk_w);
    p.lse = const_cast<float*>(lse);
    p.counts = const_cast<int32_t*>(counts);
    p.seq_tokens = const_cast<int32_t*>(seq_tokens);
    p.d_topk_w = d_topk_w;
    p.d_losses = d_losses;
    p.d_logits = d_logits;
    return launched(ep::launch_route_backward(p, num_sms, reinterpret_cast<cudaStream_t>(stream)),
                    "route backward launch");
}

size_t ep_w4_bytes(const ep_w4_t* w) {
    if (check_w4(w) != EP_OK) return (size_t)-1;
    return ep::w4_bytes({w->E, w->N, w->K, w->group, w->paired});
}

ep_status_t ep_w4_pack(const ep_w4_t* w, const uint8_t* codes, const void* scales, void* packed, ep_stream_t stream) {
    ep_status_t st = check_w4(w);
    if (st != EP_OK) return st;
    if (codes == nullptr || scales == nullptr || packed == nullptr)
        return fail(EP_ERR_INVALID_ARG, "codes / scales / packed is NULL");
    if ((reinterpret_cast<uintptr_t>(codes) & 3u) || (reinterpret_cast<uintptr_t>(scales) & 1u) || !aligned16(packed))
        return fail(EP_ERR_INVALID_ARG, "codes must be 4-byte, scales 2-byte and packed 16-byte aligned");
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;
    return launched(ep::launch_w4_pack({w->E, w->N, w->K, w->group, w->paired}, codes, scales, packed,
                                       reinterpret_cast<cudaStream_t>(stream)), "w4 pack launch");
}

ep_status_t ep_expert_w4(const ep_w4_t* w, const void* packed, int32_t mode, int32_t capacity, int64_t R,
                         int64_t max_rows, const int32_t* counts, const int32_t* offsets, const void* x,
                         const void* x_scales, int32_t payload, void* y, uint32_t* err_flags, ep_stream_t stream) {
    ep_status_t st = check_w4(w);
    if (st != EP_OK) return st;
    if (payload != EP_PAYLOAD_BF16 && payload != EP_PAYLOAD_FP8_E4M3 && payload != EP_PAYLOAD_FP8_E4M3_UE8M0)
        return fail(EP_ERR_INVALID_ARG, "payload = %d is not a payload format", payload);
    const bool fp8 = payload != EP_PAYLOAD_BF16;
    const bool ue8m0 = payload == EP_PAYLOAD_FP8_E4M3_UE8M0;
    if (fp8 && w->K % 128 != 0) return fail(EP_ERR_INVALID_ARG, "fp8 rows need K %% 128 == 0 (K = %d)", w->K);
    if (mode != EP_LAYOUT_PACKED && mode != EP_LAYOUT_CAPACITY)
        return fail(EP_ERR_INVALID_ARG, "mode = %d is not a layout mode", mode);
    if (R < 0 || max_rows < 0) return fail(EP_ERR_INVALID_ARG, "R and max_rows must not be negative");
    if (R > INT32_MAX) return fail(EP_ERR_UNSUPPORTED, "R = %lld exceeds 2^31-1", (long long)R);
    if (mode == EP_LAYOUT_CAPACITY && (capacity < 1 || R < (int64_t)w->E * capacity))
        return fail(EP_ERR_INVALID_ARG, "capacity = %d needs at least 1 and R >= E*capacity", capacity);
    if (max_rows > R) max_rows = R;
    if (max_rows == 0) return ok();
    if (mode == EP_LAYOUT_CAPACITY ? counts == nullptr : offsets == nullptr && w->E != 1)
        return fail(EP_ERR_INVALID_ARG, "counts (capacity mode) / offsets (packed) is NULL");
    if (packed == nullptr || x == nullptr || y == nullptr) return fail(EP_ERR_INVALID_ARG, "packed / x / y is NULL");
    if (!aligned16(packed) || !aligned16(x) || !aligned16(y))
        return fail(EP_ERR_INVALID_ARG, "packed, x and y must be 16-byte aligned");
    if (fp8 && (x_scales == nullptr || (!ue8m0 && (reinterpret_cast<uintptr_t>(x_scales) & 3u))))
        return fail(EP_ERR_INVALID_ARG, "fp8 rows need x_scales (4-byte aligned for f32 scales)");
    ep::W4Params p{};
    p.w = {w->E, w->N, w->K, w->group, w->paired};
    if (!ep::w4_fits(p.w, max_rows, fp8 ? 1 : 0))
        return fail(EP_ERR_UNSUPPORTED, "K = %d or max_rows = %lld is too large", w->K, (long long)max_rows);
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;
    p.packed = packed;
    p.x = x;
    p.x_scales = fp8 ? x_scales : nullptr;
    p.counts = counts;
    p.offsets = offsets;
    p.y = y;
    p.err_flags = err_flags;
    p.R = R;
    p.max_rows = max_rows;
    p.mode = mode;
    p.capacity = capacity;
    p.fp8 = fp8 ? 1 : 0;
    p.ue8m0 = ue8m0 ? 1 : 0;
    return launched(ep::launch_expert_w4(p, num_sms, reinterpret_cast<cudaStream_t>(stream)), "expert w4 launch");
}

ep_status_t ep_block_norm(const ep_norm_t* norm, const void* h, int64_t ld_h, const void* y, int64_t ld_y,
                          const float* w_post, const float* gate, const float* res_scale, const float* w_pre,
                          void* h_out, void* n, float* rstd, ep_stream_t stream) {
    ep_status_t st = check_norm(norm);
    if (st != EP_OK) return st;
    if (norm->T == 0) return ok();
    st = check_norm_inputs(norm, h, ld_h, y, ld_y, w_post, gate, w_pre);
    if (st != EP_OK) return st;
    if ((n != nullptr) != (w_pre != nullptr)) return fail(EP_ERR_INVALID_ARG, "n and w_pre go together");
    if (n == nullptr && h_out == nullptr) return fail(EP_ERR_INVALID_ARG, "h_out and n are both NULL");
    if (!aligned16(h_out) || !aligned16(n)) return fail(EP_ERR_INVALID_ARG, "h_out and n must be 16-byte aligned");
    if (h == h_out && ld_h != norm->H) return fail(EP_ERR_INVALID_ARG, "h_out in place of h needs ld_h = H");
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;

    ep::NormParams p{};
    p.h = h;
    p.y = y;
    p.w_post = w_post;
    p.gate = gate;
    p.res_scale = res_scale;
    p.w_pre = w_pre;
    p.h_out = h_out;
    p.n = n;
    p.rstd = rstd;
    p.ld_h = ld_h;
    p.ld_y = ld_y;
    p.T = norm->T;
    p.H = norm->H;
    p.f32 = norm->stream_type == EP_TYPE_F32 ? 1 : 0;
    p.gate_kind = norm->gate_kind;
    p.eps = norm->eps;
    return launched(ep::launch_block_norm(p, num_sms, reinterpret_cast<cudaStream_t>(stream)), "block norm launch");
}

size_t ep_block_norm_workspace_bytes(const ep_norm_t* norm) {
    if (check_norm(norm) != EP_OK) return (size_t)-1;
    return ep::norm_workspace_bytes(norm->T, norm->H);
}

ep_status_t ep_block_norm_backward(const ep_norm_t* norm, const void* h, int64_t ld_h, const void* y, int64_t ld_y,
                                   const float* w_post, const float* gate, const float* res_scale,
                                   const float* w_pre, const float* rstd, const void* d_h_out, const void* d_n,
                                   void* d_h, void* d_y, float* d_w_post, float* d_gate, float* d_res_scale,
                                   float* d_w_pre, void* workspace, size_t workspace_bytes, uint32_t* err_flags,
                                   ep_stream_t stream) {
    ep_status_t st = check_norm(norm);
    if (st != EP_OK) return st;
    if (norm->T > 0) {
        st = check_norm_inputs(norm, h, ld_h, y, ld_y, w_post, gate, w_pre);
        if (st != EP_OK) return st;
        if ((w_post != nullptr || w_pre != nullptr) && rstd == nullptr) return fail(EP_ERR_INVALID_ARG, "rstd is NULL");
        if (d_h == nullptr || (d_y != nullptr) != (y != nullptr))
            return fail(EP_ERR_INVALID_ARG, "d_h is NULL, or d_y does not go with y");
        if ((d_n != nullptr) != (w_pre != nullptr)) return fail(EP_ERR_INVALID_ARG, "d_n and w_pre go together");
        if (d_n == nullptr && d_h_out == nullptr) return fail(EP_ERR_INVALID_ARG, "d_h_out and d_n are both NULL");
        if (!aligned16(d_h_out) || !aligned16(d_n) || !aligned16(d_h) || !aligned16(d_y))
            return fail(EP_ERR_INVALID_ARG, "d_h_out, d_n, d_h and d_y must be 16-byte aligned");
        const size_t need = ep::norm_workspace_bytes(norm->T, norm->H);
        if (workspace == nullptr || workspace_bytes < need)
            return fail(EP_ERR_INVALID_ARG, "workspace of %zu bytes given, %zu needed", workspace_bytes, need);
        if (!aligned16(workspace)) return fail(EP_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
    }
    if ((d_w_post != nullptr) != (w_post != nullptr) || (d_w_pre != nullptr) != (w_pre != nullptr) ||
        (d_gate != nullptr) != (gate != nullptr) || (d_res_scale != nullptr) != (res_scale != nullptr))
        return fail(EP_ERR_INVALID_ARG, "each of d_w_post, d_w_pre, d_gate and d_res_scale goes with its input");
    if ((gate != nullptr) != (norm->gate_kind != EP_GATE_NONE))
        return fail(EP_ERR_INVALID_ARG, "gate and gate_kind = %d do not agree", norm->gate_kind);
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;

    ep::NormParams p{};
    p.h = h;
    p.y = y;
    p.w_post = w_post;
    p.gate = gate;
    p.res_scale = res_scale;
    p.w_pre = w_pre;
    p.rstd = const_cast<float*>(rstd);
    p.d_h_out = d_h_out;
    p.d_n = d_n;
    p.d_h = d_h;
    p.d_y = d_y;
    p.d_w_post = d_w_post;
    p.d_gate = d_gate;
    p.d_res_scale = d_res_scale;
    p.d_w_pre = d_w_pre;
    p.partial = static_cast<float*>(workspace);
    p.err_flags = err_flags;
    p.ld_h = ld_h;
    p.ld_y = ld_y;
    p.T = norm->T;
    p.H = norm->H;
    p.f32 = norm->stream_type == EP_TYPE_F32 ? 1 : 0;
    p.gate_kind = norm->gate_kind;
    p.eps = norm->eps;
    return launched(ep::launch_block_norm_backward(p, num_sms, reinterpret_cast<cudaStream_t>(stream)),
                    "block norm backward launch");
}

ep_status_t ep_dropout(int64_t T, int64_t H, int32_t type, const void* x, int64_t ld_x, const void* residual, int64_t ld_res,
                       double p, const int64_t* rng, uint64_t site, void* y, int64_t ld_y, ep_stream_t stream) {
    ep::DropoutParams d{};
    ep_status_t st = set_dropout(&d.drop, p, rng, site);
    if (st != EP_OK) return st;
    if (T < 0 || H < 1) return fail(EP_ERR_INVALID_ARG, "T = %lld must be at least 0 and H = %lld at least 1", (long long)T, (long long)H);
    if (T > INT32_MAX || H > INT32_MAX) return fail(EP_ERR_UNSUPPORTED, "T = %lld or H = %lld exceeds 2^31-1", (long long)T, (long long)H);
    if (type != EP_TYPE_BF16 && type != EP_TYPE_F32) return fail(EP_ERR_INVALID_ARG, "type = %d is not a type", type);
    if (T == 0) return ok();
    if (x == nullptr || y == nullptr) return fail(EP_ERR_INVALID_ARG, "x / y is NULL");
    if (ld_x < H || ld_y < H || (residual != nullptr && ld_res < H)) return fail(EP_ERR_INVALID_ARG, "rows are less than H = %lld apart", (long long)H);
    if ((x == y && ld_x != ld_y) || (residual == y && ld_res != ld_y))
        return fail(EP_ERR_INVALID_ARG, "y in place of an input needs rows as far apart");
    const uintptr_t mask = type == EP_TYPE_F32 ? 3u : 1u;
    if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) | reinterpret_cast<uintptr_t>(y)) & mask)
        return fail(EP_ERR_INVALID_ARG, "x, residual or y is not aligned to its elements");
    if (T * H > (int64_t)1 << 40) return fail(EP_ERR_UNSUPPORTED, "%lld rows of %lld elements are too many", (long long)T, (long long)H);
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;
    d.x = x;
    d.residual = residual;
    d.y = y;
    d.T = T;
    d.H = H;
    d.ld_x = ld_x;
    d.ld_res = ld_res;
    d.ld_y = ld_y;
    d.f32 = type == EP_TYPE_F32 ? 1 : 0;
    return launched(ep::launch_dropout(d, num_sms, reinterpret_cast<cudaStream_t>(stream)), "dropout launch");
}

ep_status_t ep_layer_norm(const ep_layer_norm_t* norm, const void* h, int64_t ld_h, const void* y, int64_t ld_y, const float* w,
                          const float* b, const int64_t* rng, void* h_out, void* n, float* stats, uint32_t* err_flags,
                          ep_stream_t stream) {
    ep_status_t st = check_layer_norm(norm);
    if (st != EP_OK) return st;
    ep::LayerNormParams p{};
    st = set_dropout(&p.drop, norm->p, rng, norm->site);
    if (st != EP_OK) return st;
    if (norm->T == 0) return ok();
    if (h == nullptr || n == nullptr) return fail(EP_ERR_INVALID_ARG, "h / n is NULL");
    if ((h_out != nullptr) != (y != nullptr)) return fail(EP_ERR_INVALID_ARG, "h_out and y go together");
    st = check_norm_rows("h", h, ld_h, norm->H);
    if (st != EP_OK) return st;
    if (y != nullptr) {
        st = check_norm_rows("y", y, ld_y, norm->H);
        if (st != EP_OK) return st;
    }
    if (!aligned16(w) || !aligned16(b) || !aligned16(h_out) || !aligned16(n))
        return fail(EP_ERR_INVALID_ARG, "w, b, h_out and n must be 16-byte aligned");
    if (h == h_out && ld_h != norm->H) return fail(EP_ERR_INVALID_ARG, "h_out in place of h needs ld_h = H");
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;
    if (y == nullptr) p.drop = ep::Dropout{};
    p.h = h;
    p.y = y;
    p.w = w;
    p.b = b;
    p.h_out = h_out;
    p.n = n;
    p.stats = stats;
    p.err_flags = err_flags;
    p.ld_h = ld_h;
    p.ld_y = ld_y;
    p.T = norm->T;
    p.H = norm->H;
    p.f32 = norm->stream_type == EP_TYPE_F32 ? 1 : 0;
    p.eps = norm->eps;
    return launched(ep::launch_layer_norm(p, num_sms, reinterpret_cast<cudaStream_t>(stream)), "layer norm launch");
}

size_t ep_layer_norm_workspace_bytes(const ep_layer_norm_t* norm) {
    if (check_layer_norm(norm) != EP_OK) return (size_t)-1;
    return ep::layer_norm_workspace_bytes(norm->T, norm->H);
}

ep_status_t ep_layer_norm_backward(const ep_layer_norm_t* norm, const void* h_out, int64_t ld_h, const float* w, const int64_t* rng,
                                   const float* stats, const void* d_h_out, const void* d_n, void* d_h, void* d_y, float* d_w,
                                   float* d_b, void* workspace, size_t workspace_bytes, uint32_t* err_flags, ep_stream_t stream) {
    ep_status_t st = check_layer_norm(norm);
    if (st != EP_OK) return st;
    ep::LayerNormParams p{};
    st = set_dropout(&p.drop, norm->p, rng, norm->site);
    if (st != EP_OK) return st;
    if (norm->T > 0) {
        if (h_out == nullptr || stats == nullptr || d_n == nullptr || d_h == nullptr)
            return fail(EP_ERR_INVALID_ARG, "h_out / stats / d_n / d_h is NULL");
        st = check_norm_rows("h", h_out, ld_h, norm->H);
        if (st != EP_OK) return st;
        if (!aligned16(w) || !aligned16(d_h_out) || !aligned16(d_n) || !aligned16(d_h) || !aligned16(d_y))
            return fail(EP_ERR_INVALID_ARG, "w, d_h_out, d_n, d_h and d_y must be 16-byte aligned");
        if (d_h == h_out && ld_h != norm->H) return fail(EP_ERR_INVALID_ARG, "d_h in place of h_out needs ld_h = H");
        const size_t need = ep::layer_norm_workspace_bytes(norm->T, norm->H);
        if (workspace == nullptr || workspace_bytes < need)
            return fail(EP_ERR_INVALID_ARG, "workspace of %zu bytes given, %zu needed", workspace_bytes, need);
        if (!aligned16(workspace)) return fail(EP_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
    }
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;
    p.h = h_out;
    p.w = w;
    p.stats = const_cast<float*>(stats);
    p.d_n = d_n;
    p.d_h_out = d_h_out;
    p.d_h = d_h;
    p.d_y = d_y;
    p.d_w = d_w;
    p.d_b = d_b;
    p.partial = static_cast<float*>(workspace);
    p.err_flags = err_flags;
    p.ld_h = ld_h;
    p.T = norm->T;
    p.H = norm->H;
    p.f32 = norm->stream_type == EP_TYPE_F32 ? 1 : 0;
    p.eps = norm->eps;
    return launched(ep::launch_layer_norm_backward(p, num_sms, reinterpret_cast<cudaStream_t>(stream)), "layer norm backward launch");
}

ep_status_t ep_quant_i8(int32_t E, int32_t K, int32_t mode, int32_t capacity, int64_t R, const int32_t* counts,
                        const int32_t* offsets, const void* x, int64_t ld_x, int8_t* q, float* scales, uint32_t* err_flags,
                        ep_stream_t stream) {
    if (E < 1) return fail(EP_ERR_INVALID_ARG, "E = %d < 1", E);
    if (E > EP_MAX_EXPERTS) return fail(EP_ERR_UNSUPPORTED, "E = %d > %d", E, EP_MAX_EXPERTS);
    if (K <= 0 || K % 16 != 0) return fail(EP_ERR_INVALID_ARG, "K = %d must be a positive multiple of 16", K);
    if (K > EP_MAX_QUANT_WIDTH) return fail(EP_ERR_UNSUPPORTED, "K = %d > %d", K, EP_MAX_QUANT_WIDTH);
    ep_status_t st = check_rows(E, mode, capacity, R, counts, offsets, true);
    if (st != EP_OK) return st;
    if (R == 0) return ok();
    if (x == nullptr || q == nullptr || scales == nullptr) return fail(EP_ERR_INVALID_ARG, "x / q / scales is NULL");
    if (ld_x < K || ld_x % 8 != 0) return fail(EP_ERR_INVALID_ARG, "ld_x = %lld must be a multiple of 8 and at least K = %d", (long long)ld_x, K);
    if (!aligned16(x) || !aligned16(q) || (reinterpret_cast<uintptr_t>(scales) & 3u))
        return fail(EP_ERR_INVALID_ARG, "x and q must be 16-byte, scales 4-byte aligned");
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;
    ep::QuantParams p{};
    p.x = x;
    p.counts = counts;
    p.offsets = offsets;
    p.q = q;
    p.scales = scales;
    p.err_flags = err_flags;
    p.R = R;
    p.ld = ld_x;
    p.E = E;
    p.K = K;
    p.mode = mode;
    p.capacity = capacity;
    return launched(ep::launch_quant_i8(p, num_sms, reinterpret_cast<cudaStream_t>(stream)), "quant i8 launch");
}

size_t ep_i8_bytes(const ep_i8_t* w) {
    if (check_i8(w) != EP_OK) return (size_t)-1;
    return ep::i8_bytes({w->E, w->N, w->K, w->paired});
}

ep_status_t ep_i8_pack(const ep_i8_t* w, const int8_t* codes, const float* scales, void* packed, ep_stream_t stream) {
    ep_status_t st = check_i8(w);
    if (st != EP_OK) return st;
    if (codes == nullptr || scales == nullptr || packed == nullptr)
        return fail(EP_ERR_INVALID_ARG, "codes / scales / packed is NULL");
    if (!aligned16(codes) || (reinterpret_cast<uintptr_t>(scales) & 3u) || !aligned16(packed))
        return fail(EP_ERR_INVALID_ARG, "codes and packed must be 16-byte, scales 4-byte aligned");
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;
    return launched(ep::launch_i8_pack({w->E, w->N, w->K, w->paired}, codes, scales, packed, reinterpret_cast<cudaStream_t>(stream)),
                    "i8 pack launch");
}

ep_status_t ep_expert_i8(const ep_i8_t* w, const void* packed, int32_t mode, int32_t capacity, int64_t R, int64_t max_rows,
                         const int32_t* counts, const int32_t* offsets, const int8_t* x, const float* x_scales, void* y,
                         uint32_t* err_flags, ep_stream_t stream) {
    ep_status_t st = check_i8(w);
    if (st != EP_OK) return st;
    if (max_rows < 0) return fail(EP_ERR_INVALID_ARG, "max_rows must not be negative");
    if (max_rows > R) max_rows = R;
    st = check_rows(w->E, mode, capacity, R, counts, offsets, w->E == 1 || max_rows == 0);
    if (st != EP_OK) return st;
    if (max_rows == 0) return ok();
    if (packed == nullptr || x == nullptr || x_scales == nullptr || y == nullptr)
        return fail(EP_ERR_INVALID_ARG, "packed / x / x_scales / y is NULL");
    if (!aligned16(packed) || !aligned16(x) || !aligned16(y) || (reinterpret_cast<uintptr_t>(x_scales) & 3u))
        return fail(EP_ERR_INVALID_ARG, "packed, x and y must be 16-byte, x_scales 4-byte aligned");
    ep::I8Params p{};
    p.w = {w->E, w->N, w->K, w->paired};
    if (!ep::i8_fits(p.w, max_rows)) return fail(EP_ERR_UNSUPPORTED, "max_rows = %lld is too large", (long long)max_rows);
    int num_sms = 0;
    st = device_info(&num_sms);
    if (st != EP_OK) return st;
    p.packed = packed;
    p.x = x;
    p.x_scales = x_scales;
    p.counts = counts;
    p.offsets = offsets;
    p.y = y;
    p.err_flags = err_flags;
    p.R = R;
    p.max_rows = max_rows;
    p.mode = mode;
    p.capacity = capacity;
    return launched(ep::launch_expert_i8(p, num_sms, reinterpret_cast<cudaStream_t>(stream)), "expert i8 launch");
}

}  // extern "C"
