// vocab.h -- the vocabulary's two ends: embedding lookup and its gradient,
// the head's cross entropy and its gradient (host launch interface).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gr {

struct EmbedLookupArgs {
    const int32_t* tokens;  // [n]
    int32_t n, V, D;
    float scale;
    const void* weight;  // [V] rows of D elements, wstride apart
    int64_t wstride;
    void* out;           // [n] rows, ostride apart
    int64_t ostride;
};

struct EmbedBackwardArgs {
    const int32_t* tokens;  // [n]
    int32_t n, V, D;
    float scale;
    const void* grad;    // [n] rows of D elements, gstride apart
    int64_t gstride;
    void* gweight;       // [V] rows, wstride apart
    int64_t wstride;
    int32_t accumulate;
};

// The head's workspace: what a handle of `max_rows` rows needs.
struct HeadArgs {
    int32_t N, V, D;
    float scale;
    const void* hidden;  // [N] rows of D elements, hstride apart
    int64_t hstride;
    const void* weight;  // [V] rows, wstride apart
    int64_t wstride;
    const int32_t* targets;  // [N]
    float* loss;             // [N] out
    float* lse;              // [N] out (forward) / in (backward)
    const float* grad_loss;  // [N]
    void* ghidden;           // [N] rows, ghstride apart, or nullptr
    int64_t ghstride;
    void* gweight;           // [V] rows, gwstride apart, or nullptr
    int64_t gwstride;
    int32_t accumulate;
    // workspace
    float2* parts;   // [tiles][N] max and sum of exp(z - max) of a row's tile
    float* zt;       // [N] the target's logit
    float* G;        // [N][Vp] a piece of the logits' gradient
    int32_t Vp;      // words of a piece
    float* gh_acc;   // [N][D] sums of grad_hidden over the pieces
};

constexpr int kHeadTile = 64;

hipError_t launch_embed_lookup(const EmbedLookupArgs& a, int dtype, hipStream_t st);
hipError_t launch_embed_backward(const EmbedBackwardArgs& a, int dtype, hipStream_t st);
hipError_t launch_head_loss(const HeadArgs& a, int dtype, hipStream_t st);
hipError_t launch_head_backward(const HeadArgs& a, int dtype, hipStream_t st);

}  // namespace gr
