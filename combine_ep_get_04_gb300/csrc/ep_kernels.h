// ep_kernels.h -- host-side launchers of the dispatch / combine kernels and
// their parameter blocks (internal to the library; the public C ABI is
// include/ep.h).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace ep {

// Launches `kern`; with pdl, under programmatic stream serialization: it may
// begin while the previous kernel of the stream finishes, and waits
// (pdl_wait) before it writes global memory or reads what that kernel may
// write (before the wait it only prefetches into L2, and reads such memory
// only as an address hint for a prefetch).  Used for latency-sized grids
// (about one unit of work per CTA), where the launch gap is a large share of
// the time; large persistent grids launch normally.
// With cluster > 1, that many consecutive CTAs form a cluster.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(bool pdl, int cluster, void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                            cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_kernel(bool pdl, void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                          cudaStream_t stream, Args&&... args) {
    return launch_clusters(pdl, 1, kern, grid, block, smem, stream, args...);
}

// Sets the text ep_last_error() returns on the calling thread.
void record_last_error(const char* msg);

// ----------------------------------------------------------------- layout

constexpr int64_t kLayoutChunk = 1024;   // entries ranked by one CTA
constexpr int64_t kLayoutSmallN = 4096;  // up to this many entries: one launch, no workspace

struct LayoutParams {
    const int32_t* topk_idx;
    int32_t* counts;
    int32_t* offsets;
    int32_t* part_counts;
    int32_t* part_offsets;
    int32_t* slot_of;
    int32_t* src_token;
    int32_t* src_k;
    int32_t* hist;        // [num_chunks][E] workspace, or nullptr for the one-launch path
    uint32_t* err_flags;  // may be nullptr
    int64_t N;            // T * k
    int64_t R;            // receive rows
    int64_t chunk;        // set by launch_layout
    int num_chunks;       // set by launch_layout
    int E, P, k, mode, cap;
};

int64_t layout_num_chunks(int64_t N);
bool layout_uses_workspace(int64_t N);
size_t layout_workspace_bytes(int64_t N, int E);
size_t layout_rank_smem_bytes(int E);
cudaError_t launch_layout(const LayoutParams& p, int num_sms, cudaStream_t stream);

// --------------------------------------------------------------- dispatch

struct DispatchParams {
    const void* x;          // bf16 [T, H]
    const float* topk_w;    // [T, k] or nullptr
    const int32_t* slot_of; // [T, k]
    void* recv;             // bf16 or e4m3 [R, H]
    void* recv_scales;      // [R, H/128] f32, or u8 exponents with ue8m0 (fp8)
    float* recv_w;          // [R] or nullptr
    uint32_t* err_flags;    // may be nullptr
    int64_t R;              // receive rows
    int T, H, k;
    int ue8m0;              // power-of-two scales stored as exponent bytes
};

cudaError_t launch_dispatch_bf16(const DispatchParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_dispatch_fp8(const DispatchParams& p, int num_sms, cudaStream_t stream);

// ------------------------------------------------ layout + dispatch fused

constexpr int64_t kFusedMaxN = 2048;   // routing entries: every CTA counts them all
constexpr int64_t kFusedMaxT = 2048;

struct FusedLaunch {
    const int32_t* topk_idx;
    const void* x;
    const float* topk_w;
    int32_t* counts;
    int32_t* offsets;
    int32_t* part_counts;
    int32_t* part_offsets;
    int32_t* slot_of;
    int32_t* src_token;
    int32_t* src_k;
    void* recv;
    void* recv_scales;
    float* recv_w;
    uint32_t* err_flags;
    int64_t R;
    int T, H, E, k, P, mode, cap, fp8, ue8m0;
};

bool fused_layout_dispatch_fits(int64_t N, int64_t T, int E);
cudaError_t launch_layout_dispatch(const FusedLaunch& f, int num_sms, cudaStream_t stream);

// ---------------------------------------------------------------- combine

struct CombineParams {
    const void* y;          // bf16 [R, H], or e4m3 [R, H] with fp8
    const void* y_scales;   // fp8: [R, H/128] f32, or u8 exponents with ue8m0
    int fp8, ue8m0;
    const float* topk_w;    // [T, k]
    const int32_t* slot_of; // [T, k]
    void* out;              // bf16 [T, H]
    uint32_t* err_flags;    // may be nullptr
    int64_t R;              // rows of y
    int T, H, k;
};

cudaError_t launch_combine(const CombineParams& p, int num_sms, cudaStream_t stream);

// The combine addressed by the expert-side maps: base carries y, scales,
// out, err_flags and the shape (its slot_of / topk_w are ignored).
struct CombineSrcParams {
    CombineParams base;
    const float* row_w;       // [R] or nullptr (unweighted)
    const int32_t* src_token; // [R], -1 = no copy
    const int32_t* src_k;     // [R]
    void* workspace;          // combine_src_workspace_bytes(T, k) bytes
};

// Bytes of one [T, k] map rounded up to 256; the workspace holds two.
size_t combine_src_map_bytes(int64_t T, int k);
inline size_t combine_src_workspace_bytes(int64_t T, int k) { return 2 * combine_src_map_bytes(T, k); }

cudaError_t launch_combine_src(const CombineSrcParams& p, int num_sms, cudaStream_t stream);

// ------------------------------------------------------------------ route

struct RouteParams {
    const void* logits;          // [T, E], rows ld apart
    const float* select_bias;    // [E] or nullptr
    const uint8_t* token_mask;   // [T] or nullptr
    const int32_t* seq_offsets;  // [S + 1], or nullptr: one sequence
    int32_t* topk_idx;           // [T, k]; written forward, read backward, as the next five
    float* topk_w;               // [T, k]
    float* lse;                  // [T] or nullptr
    int32_t* counts;             // [S, E]
    float* prob_sums;            // [S, E]
    int32_t* seq_tokens;         // [S + 2]
    float* losses;               // [2], or nullptr: the choice alone
    const float* d_topk_w;       // backward
    const float* d_losses;
    void* d_logits;
    // workspace, one row for each run of `chunk` tokens of one sequence
    float* part_prob;            // [runs, E]
    int32_t* part_count;         // [runs, E]
    float* part_z;               // [runs]
    int32_t* part_live;          // [runs]
    float* part_loss;            // [S, expert blocks]
    float* seq_z;                // [S]
    uint32_t* ticket;
    uint32_t* err_flags;
    int64_t ld;
    int T, E, k, groups, topk_groups, full_softmax, f32, S;
    int chunk, per_group, wide;  // set by the launchers; wide: rows are read and written by wide accesses
    float balance_coef, z_coef;
};

// Splits the workspace over the part_* members (base may be nullptr); returns its size.
size_t route_workspace(RouteParams* p, void* base);
cudaError_t launch_route(const RouteParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_route_backward(const RouteParams& p, int num_sms, cudaStream_t stream);

// -------------------------------------------------------------- expert w4

struct W4Shape {
    int E, N, K, group, paired;
};

struct W4Params {
    W4Shape w;
    const void* packed;
    const void* x;
    const void* x_scales;      // f32 or UE8M0 bytes (fp8)
    const int32_t* counts;
    const int32_t* offsets;
    void* y;
    uint32_t* err_flags;
    int64_t R, max_rows;
    int mode, capacity, fp8, ue8m0;
};

size_t w4_bytes(const W4Shape& w);
bool w4_packs(const W4Shape& w);                                // whether one launch packs them
bool w4_fits(const W4Shape& w, int64_t max_rows, int fp8);      // whether one launch covers the rows
cudaError_t launch_w4_pack(const W4Shape& w, const uint8_t* codes, const void* scales, void* packed, cudaStream_t stream);
cudaError_t launch_expert_w4(const W4Params& p, int num_sms, cudaStream_t stream);

// ------------------------------------------------------------- block norm

struct NormParams {
    const void* h;             // stream type [T, H], rows ld_h apart
    const void* y;             // bf16 [T, H], rows ld_y apart, or nullptr
    const float* w_post;       // [H] or nullptr
    const float* gate;         // [H] or [T] by gate_kind, or nullptr
    const float* res_scale;    // [1] or nullptr
    const float* w_pre;        // [H] or nullptr
    void* h_out;               // stream type [T, H] or nullptr (forward)
    void* n;                   // bf16 [T, H] or nullptr (forward)
    float* rstd;               // [2, T]; written forward (may be nullptr), read backward
    const void* d_h_out;       // backward from here on
    const void* d_n;
    void* d_h;
    void* d_y;
    float* d_w_post;
    float* d_gate;
    float* d_res_scale;
    float* d_w_pre;
    float* partial;            // workspace: column sums of each group of CTAs, then each CTA's d_res_scale
    uint32_t* err_flags;       // may be nullptr
    int64_t ld_h, ld_y;
    int T, H;
    int f32;                   // stream type
    int gate_kind;             // EP_GATE_*
    float eps;
};

size_t norm_workspace_bytes(int T, int H);
cudaError_t launch_block_norm(const NormParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_block_norm_backward(const NormParams& p, int num_sms, cudaStream_t stream);

}  // namespace ep
