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

constexpr int kEmbedFew = 512;    // at most so many tokens: no sort
constexpr int kSortFew = 2048;    // at most so many: sorted by one workgroup
constexpr int kSortBits = 11;     // of a sort pass at most
constexpr int kSortChunk = 1024;  // positions of a sort workgroup
constexpr int kSumTiles = 8192;   // tiles of the sums at most

struct EmbedPlan {
    int32_t passes, bits, blocks;  // of the sort
    int32_t tile, tiles;           // of the sums
};

// lanes: threads to a row in the sums
EmbedPlan embed_plan(int64_t n, int64_t vocab, int lanes);

// The gradient's workspace (device).
struct EmbedSpace {
    int32_t* keys[2];  // [n] words in sorted order, by turns
    int32_t* pos[2];   // [n] their positions
    int32_t* table;    // [workgroups][digits] counts
    int32_t* totals;   // [digits]
    float* parts;      // [tiles][2][Dp] sums of words that cross tiles
};

struct EmbedBackwardArgs {
    const int32_t* tokens;  // [n]
    int32_t n, V, D, Dp;    // Dp: D rounded up to 8
    float scale;
    const void* grad;    // [n] rows of D elements, gstride apart
    int64_t gstride;
    void* gweight;       // [V] rows, wstride apart
    int64_t wstride;
    int32_t accumulate;
    EmbedSpace ws;
};

// Sizes of a head's workspace, fixed at init for its most rows.
struct HeadPlan {
    int32_t planes;    // bf16 planes of an element: 1 (bf16) or 3 (fp32)
    int32_t halves;    // fp16 planes of an element for the logits: 0 (bf16) or 2 (fp32)
    int32_t Dp;        // dim rounded up to 8
    int32_t part_rows; // rows of one forward pass (more go in several)
    int32_t Vg;        // words of a piece of the backward
    int32_t Vw;        // words of a packed piece of the table
    int64_t packed, parts, G, gh, gw, W;  // elements of the buffers below
};

HeadPlan head_plan(int64_t max_rows, int64_t vocab, int64_t dim, int dtype, bool backward);

// The workspace (device): rows that have a target are packed, in order.
struct HeadSpace {
    int32_t* count;    // [1] rows with a target
    int32_t* target;   // [packed row] its target
    int32_t* source;   // [packed row] its row
    int32_t* place;    // [row] its packed row, -1 without a target
    float* gscale;     // [packed row] scale * grad_loss
    float* lse;        // [packed row]
    float* zt;         // [packed row] the target's logit
    uint16_t* H;       // [planes][rows][Dp] packed hidden states
    uint16_t* Hh;      // [halves][rows][Dp] the same, scaled row by row
    float* hdown;      // [packed row] what divides the row's scale out
    uint16_t* Wh;      // [halves][Vw][Dp] a piece of the table, scaled word by word
    float* wdown;      // [Vw] what divides a word's scale out
    float2* parts;     // [parts of the vocabulary][rows] max and sum of 2^(y - max), y = z log2 e
    uint16_t* W;       // [planes][Vw][Dp] a piece of the table, where it cannot be read as it lies
    uint16_t* G;       // [planes][rows][Vg] a piece of the logits' gradient
    float* gh;         // [splits][rows][Dp] partial sums of grad_hidden
    float* gw;         // [splits][Vg][Dp] partial sums of grad_weight
};

struct HeadArgs {
    int32_t N, V, D;
    float scale;
    const void* hidden;  // [N] rows of D elements, hstride apart
    int64_t hstride;
    const void* weight;  // [V] rows, wstride apart
    int64_t wstride;
    const int32_t* targets;  // [N]
    float* loss;             // [N] out
    float* lse;              // [N] out
    const float* lse_in;     // [N] in (backward)
    const float* grad_loss;  // [N]
    void* ghidden;           // [N] rows, ghstride apart, or nullptr
    int64_t ghstride;
    void* gweight;           // [V] rows, gwstride apart, or nullptr
    int64_t gwstride;
    int32_t accumulate;
    HeadPlan plan;
    HeadSpace ws;
};

hipError_t launch_embed_lookup(const EmbedLookupArgs& a, int dtype, hipStream_t st);
hipError_t launch_embed_backward(const EmbedBackwardArgs& a, int dtype, hipStream_t st);
hipError_t launch_head_loss(const HeadArgs& a, int dtype, hipStream_t st);
hipError_t launch_head_backward(const HeadArgs& a, int dtype, hipStream_t st);

}  // namespace gr
