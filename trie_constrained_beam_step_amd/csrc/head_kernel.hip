// head_kernel.hip -- softmax cross entropy of hidden states against the head's
// table, without keeping the logits, and its gradient.
//
// With z[n][v] = scale * <h_n, w_v>:
//   forward   z in tiles; a tile leaves each of its rows' (max, sum of
//             exp(z - max)); a second kernel joins a row's tiles.
//   backward  a piece of the vocabulary at a time: z again, G = scale * g *
//             (exp(z - lse) - onehot) into the workspace, then the piece's
//             share of grad_hidden = G W and its rows of grad_weight = G^T H.
#include "device_common.h"
#include "gr.h"
#include "vocab.h"

namespace gr {
namespace {

constexpr int kT = kHeadTile;  // 64 x 64 tiles, 256 threads, 4 x 4 per thread
constexpr int kK = 16;

__device__ __forceinline__ void store_elem(float* p, int64_t i, float v) { p[i] = v; }
// bf16 with round to nearest even; NaN stays NaN
__device__ __forceinline__ void store_elem(uint16_t* p, int64_t i, float v) {
    const uint32_t b = __float_as_uint(v);
    p[i] = (v != v) ? (uint16_t)((b >> 16) | 0x40) : (uint16_t)((b + 0x7FFFu + ((b >> 16) & 1u)) >> 16);
}

__device__ __forceinline__ bool has_target(const HeadArgs& a, int n) {
    return n < a.N && a.targets[n] >= 0 && a.targets[n] < a.V;
}

// c[i][j] = sum_k A(m0 + ty*4 + i, k) * B(n0 + tx*4 + j, k), k < K
template <typename FA, typename FB>
__device__ void tile_product(int K, FA fa, FB fb, float c[4][4]) {
    __shared__ float sa[kK][kT + 1], sb[kK][kT + 1];
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) c[i][j] = 0.0f;
    for (int k0 = 0; k0 < K; k0 += kK) {
        __syncthreads();
        for (int e = threadIdx.x; e < kK * kT; e += 256) {
            const int k = e % kK, r = e / kK;
            sa[k][r] = k0 + k < K ? fa(r, k0 + k) : 0.0f;
            sb[k][r] = k0 + k < K ? fb(r, k0 + k) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < kK; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) c[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], c[i][j]);
    }
}

// logits of words v0 .. v0+63 (rows of c) and hidden states n0 .. n0+63
template <typename T>
__device__ void logits_tile(const HeadArgs& a, int v0, int n0, float c[4][4]) {
    tile_product(
        a.D,
        [&](int r, int k) { return v0 + r < a.V ? load_elem((const T*)a.weight + (int64_t)(v0 + r) * a.wstride, k) : 0.0f; },
        [&](int r, int k) {
            return has_target(a, n0 + r) ? load_elem((const T*)a.hidden + (int64_t)(n0 + r) * a.hstride, k) : 0.0f;
        },
        c);
}

template <typename T>
__global__ __launch_bounds__(256) void head_parts_kernel(HeadArgs a) {
    __shared__ float z[kT][kT + 1];
    const int v0 = blockIdx.x * kT, n0 = blockIdx.y * kT;
    float c[4][4];
    logits_tile<T>(a, v0, n0, c);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) z[tx * 4 + j][ty * 4 + i] = c[i][j] * a.scale;
    __syncthreads();
    if (threadIdx.x < kT && has_target(a, n0 + threadIdx.x)) {
        const int n = n0 + threadIdx.x, nv = min(kT, a.V - v0);
        float m = kFarBelow, s = 0.0f;
        for (int v = 0; v < nv; ++v) m = fmaxf(m, z[threadIdx.x][v]);
        for (int v = 0; v < nv; ++v) s += expf(z[threadIdx.x][v] - m);
        a.parts[(int64_t)blockIdx.x * a.N + n] = make_float2(m, s);
        const int t = a.targets[n] - v0;
        if (t >= 0 && t < nv) a.zt[n] = z[threadIdx.x][t];
    }
}

__global__ __launch_bounds__(256) void head_join_kernel(HeadArgs a, int tiles) {
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= a.N) return;
    float loss = 0.0f, lse = 0.0f;
    if (has_target(a, n)) {
        float m = kFarBelow, s = 0.0f;
        for (int i = 0; i < tiles; ++i) m = fmaxf(m, a.parts[(int64_t)i * a.N + n].x);
        for (int i = 0; i < tiles; ++i) {
            const float2 p = a.parts[(int64_t)i * a.N + n];
            s += p.y * expf(p.x - m);
        }
        lse = m + logf(s);
        loss = lse - a.zt[n];
    }
    a.loss[n] = loss;
    a.lse[n] = lse;
}

template <typename T>
__global__ __launch_bounds__(256) void head_logit_grad_kernel(HeadArgs a, int vp) {
    const int v0 = vp + blockIdx.x * kT, n0 = blockIdx.y * kT;
    float c[4][4];
    logits_tile<T>(a, v0, n0, c);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx * 4 + j;
        if (n >= a.N) continue;
        const bool ok = has_target(a, n);
        const float g = ok ? a.scale * a.grad_loss[n] : 0.0f, lse = ok ? a.lse[n] : 0.0f;
        for (int i = 0; i < 4; ++i) {
            const int v = v0 + ty * 4 + i;
            if (v >= a.V) continue;
            float p = expf(c[i][j] * a.scale - lse);
            if (ok && v == a.targets[n]) p -= 1.0f;
            a.G[(int64_t)n * a.Vp + (v - vp)] = ok ? g * p : 0.0f;
        }
    }
}

// grad_hidden[n][d] += sum over the piece's words of G[n][v] W[v][d]
template <typename T>
__global__ __launch_bounds__(256) void head_ghidden_kernel(HeadArgs a, int vp, int nv, bool first, bool last) {
    const int d0 = blockIdx.x * kT, n0 = blockIdx.y * kT;
    float c[4][4];
    tile_product(
        nv, [&](int r, int k) { return d0 + r < a.D ? load_elem((const T*)a.weight + (int64_t)(vp + k) * a.wstride, d0 + r) : 0.0f; },
        [&](int r, int k) { return n0 + r < a.N ? a.G[(int64_t)(n0 + r) * a.Vp + k] : 0.0f; }, c);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    for (int j = 0; j < 4; ++j)
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + tx * 4 + j, d = d0 + ty * 4 + i;
            if (n >= a.N || d >= a.D) continue;
            float* acc = a.gh_acc + (int64_t)n * a.D + d;
            const float s = first ? c[i][j] : *acc + c[i][j];
            if (last) store_elem((T*)a.ghidden + (int64_t)n * a.ghstride, d, has_target(a, n) ? s : 0.0f);
            else *acc = s;
        }
}

// grad_weight[v][d] = sum_n G[n][v] H[n][d]
template <typename T>
__global__ __launch_bounds__(256) void head_gweight_kernel(HeadArgs a, int vp, int nv) {
    const int d0 = blockIdx.x * kT, v0 = blockIdx.y * kT;
    float c[4][4];
    tile_product(
        a.N,
        [&](int r, int k) {
            return d0 + r < a.D && has_target(a, k) ? load_elem((const T*)a.hidden + (int64_t)k * a.hstride, d0 + r) : 0.0f;
        },
        [&](int r, int k) { return v0 + r < nv ? a.G[(int64_t)k * a.Vp + v0 + r] : 0.0f; }, c);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    for (int j = 0; j < 4; ++j)
        for (int i = 0; i < 4; ++i) {
            const int v = v0 + tx * 4 + j, d = d0 + ty * 4 + i;
            if (v >= nv || d >= a.D) continue;
            T* o = (T*)a.gweight + (int64_t)(vp + v) * a.gwstride;
            store_elem(o, d, a.accumulate ? load_elem(o, d) + c[i][j] : c[i][j]);
        }
}

unsigned tiles_of(int x) { return (unsigned)((x + kT - 1) / kT); }

template <typename T>
hipError_t head_loss_t(const HeadArgs& a, hipStream_t st) {
    head_parts_kernel<T><<<dim3(tiles_of(a.V), tiles_of(a.N)), 256, 0, st>>>(a);
    head_join_kernel<<<dim3((unsigned)((a.N + 255) / 256)), 256, 0, st>>>(a, (int)tiles_of(a.V));
    return hipGetLastError();
}

template <typename T>
hipError_t head_backward_t(const HeadArgs& a, hipStream_t st) {
    for (int vp = 0; vp < a.V; vp += a.Vp) {
        const int nv = a.V - vp < a.Vp ? a.V - vp : a.Vp;
        if (a.N) head_logit_grad_kernel<T><<<dim3(tiles_of(nv), tiles_of(a.N)), 256, 0, st>>>(a, vp);
        if (a.N && a.ghidden)
            head_ghidden_kernel<T><<<dim3(tiles_of(a.D), tiles_of(a.N)), 256, 0, st>>>(a, vp, nv, vp == 0, vp + nv == a.V);
        if (a.gweight) head_gweight_kernel<T><<<dim3(tiles_of(a.D), tiles_of(nv)), 256, 0, st>>>(a, vp, nv);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_head_loss(const HeadArgs& a, int dtype, hipStream_t st) {
    if (a.N == 0) return hipSuccess;
    return dtype == GR_BF16 ? head_loss_t<uint16_t>(a, st) : head_loss_t<float>(a, st);
}

hipError_t launch_head_backward(const HeadArgs& a, int dtype, hipStream_t st) {
    if (a.N == 0 && (a.accumulate || !a.gweight)) return hipSuccess;
    return dtype == GR_BF16 ? head_backward_t<uint16_t>(a, st) : head_backward_t<float>(a, st);
}

}  // namespace gr
