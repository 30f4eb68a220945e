// block_kernels.h -- launch declarations of the operators at the ends of a block.
#pragma once
#include "ep_kernels.h"

namespace ep {

// launch_kernel, with every `cluster` consecutive CTAs a cluster.
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
