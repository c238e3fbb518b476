// head_kernel.hip -- softmax cross entropy of hidden states against the head's
// table, without keeping the logits, and its gradient.
//
// With z[n][v] = scale * <h_n, w_v>:
//   forward   z in tiles on the matrix cores; a wave of a tile leaves, for each
//             of its rows, (max, sum of exp(z - max)) over its words: a part.
//             A second kernel joins a row's parts.
//   backward  a piece of the vocabulary at a time: z again, G = scale * g *
//             (exp(z - lse) - onehot) into the workspace, then the piece's
//             share of grad_hidden = G W and its rows of grad_weight = G^T H.
// All three products are gemm_tile.h's, with the words (first product) or the
// width (the others) as its rows m and the hidden states (or words) as its n.
//
// Rows without a target are left out at the start (pack_rows_kernel): the
// products run over the packed rows only, whose number is known on the device
// alone, so grids are sized for all rows and workgroups behind the count end
// at once.
#include "device_common.h"
#include "gemm_tile.h"
#include "gr.h"
#include "vocab.h"

namespace gr {
namespace {

__device__ __forceinline__ uint16_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ void store_elem(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store_elem(uint16_t* p, int64_t i, float v) { p[i] = bf16_bits(v); }

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Two values rounded to bf16, the first in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float x, float y) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));
}

// x and y as PL bf16 planes (gemm_tile.h), each plane's pair packed.  A value
// whose first plane would round to infinity starts from the largest finite
// bf16 and the other planes carry the rest; a NaN comes back as the rest.
template <int PL>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&out)[PL]) {
    if (PL == 1) {
        out[0] = bf16_pair(x, y);
        return;
    }
    constexpr float kMost = 3.38953139e38f;  // the largest finite bf16
    out[0] = bf16_pair(__builtin_amdgcn_fmed3f(x, -kMost, kMost), __builtin_amdgcn_fmed3f(y, -kMost, kMost));
#pragma unroll
    for (int p = 1; p < PL; ++p) {
        x -= __uint_as_float(out[p - 1] << 16);
        y -= __uint_as_float(out[p - 1] & 0xFFFF0000u);
        out[p] = bf16_pair(x, y);
    }
}

__device__ __forceinline__ bool has_target(const HeadArgs& a, int n) {
    return n < a.N && (uint32_t)a.targets[n] < (uint32_t)a.V;
}

// ------------------------------------------------------------ packing

// Elements [d, d + 8) of a row, zeros behind D.  Rows need no alignment beyond
// the element's: the hardware takes 16-byte loads anywhere.
typedef f32x4v f32x4_anywhere __attribute__((aligned(4)));
typedef u32x4 u32x4_anywhere __attribute__((aligned(2)));

__device__ __forceinline__ void load8(const float* src, int d, int D, float (&x)[8]) {
    if (d + 8 <= D) {
        const f32x4v lo = *(const f32x4_anywhere*)(src + d), hi = *(const f32x4_anywhere*)(src + d + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = lo[e], x[e + 4] = hi[e];
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = d + e < D ? src[d + e] : 0.0f;
}
__device__ __forceinline__ u32x4 load8_bits(const uint16_t* src, int d, int D) {
    if (d + 8 <= D) return *(const u32x4_anywhere*)(src + d);
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (d + e < D) v[e >> 1] |= (uint32_t)src[d + e] << (16 * (e & 1));
    return v;
}

// Row `src` of D elements into planes of Dp (a multiple of 8).
__device__ __forceinline__ void pack_row(const uint16_t* src, int D, int Dp, uint16_t* dst, int64_t, int lane, int lanes) {
    for (int d = lane * 8; d < Dp; d += lanes * 8) *(u32x4*)(dst + d) = load8_bits(src, d, D);
}
__device__ __forceinline__ void pack_row(const float* src, int D, int Dp, uint16_t* dst, int64_t plane, int lane, int lanes) {
    for (int d = lane * 8; d < Dp; d += lanes * 8) {
        float x[8];
        load8(src, d, D, x);
        u32x4 v[3];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t b[3];
            split_pair<3>(x[2 * e], x[2 * e + 1], b);
#pragma unroll
            for (int p = 0; p < 3; ++p) v[p][e] = b[p];
        }
#pragma unroll
        for (int p = 0; p < 3; ++p) *(u32x4*)(dst + p * plane + d) = v[p];
    }
}

// Row `src` scaled by a power of two into two fp16 planes (gemm_tile.h), by one
// wave; returns what divides the scale out again.
__device__ __forceinline__ float pack_row_half(const float* src, int D, int Dp, uint16_t* dst, int64_t plane, int lane) {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    float most = 0.0f;
    for (int d = lane * 8; d < Dp; d += 512) {
        float x[8];
        load8(src, d, D, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(x[e]));
    }
    most = wave_max(most);
    const int exponent = (int)((__float_as_uint(most) >> 23) & 255) - 127;
    const int up = most == 0.0f ? 0 : min(126, 14 - exponent);  // 2^14 <= most * 2^up < 2^15
    const float scale = __uint_as_float((uint32_t)(127 + up) << 23);
    for (int d = lane * 8; d < Dp; d += 512) {
        float x[8];
        load8(src, d, D, x);
        u32x4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float y0 = x[2 * e] * scale, y1 = x[2 * e + 1] * scale;
            const f16x2 h = {(_Float16)y0, (_Float16)y1};
            const f16x2 l = {(_Float16)(y0 - (float)h[0]), (_Float16)(y1 - (float)h[1])};
            hi[e] = __builtin_bit_cast(uint32_t, h);
            lo[e] = __builtin_bit_cast(uint32_t, l);
        }
        *(u32x4*)(dst + d) = hi;
        *(u32x4*)(dst + plane + d) = lo;
    }
    return __uint_as_float((uint32_t)(127 - up) << 23);
}

// what a packing kernel writes: planes as they are (bf16: one, fp32: three, for
// the gradients' products), scaled halves (fp32, for the logits)
constexpr int kPackPlanes = 1, kPackHalves = 2;

// The rows that have a target, packed in order (40,960 rows of 512 bf16: 22 us,
// 3.8 TB/s).  Each workgroup counts the
// targets before its own rows by itself (the targets of 2^16 rows are 256 KB
// of L2 reads; a scan kernel before this one would cost a launch).
template <typename T>
__global__ __launch_bounds__(256) void pack_rows_kernel(HeadArgs a, int64_t rows_cap, int rows_per_wg, int what, bool zero_rows) {
    __shared__ int wsum[4], base;
    const int r0 = blockIdx.x * rows_per_wg;
    int c = 0;
    if ((uintptr_t)a.targets % 16 == 0) {  // r0 is a multiple of 4
        typedef int i32x4 __attribute__((ext_vector_type(4)));
#pragma unroll 4
        for (int i = threadIdx.x * 4; i < r0; i += 1024) {
            const i32x4 t = *(const i32x4*)(a.targets + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) c += (uint32_t)t[e] < (uint32_t)a.V ? 1 : 0;
        }
    } else {
        for (int i = threadIdx.x; i < r0; i += 256) c += (uint32_t)a.targets[i] < (uint32_t)a.V ? 1 : 0;
    }
    c = (int)wave_sum_ll(c);
    if ((threadIdx.x & 63) == 0) wsum[threadIdx.x >> 6] = c;
    __syncthreads();
    if (threadIdx.x == 0) base = wsum[0] + wsum[1] + wsum[2] + wsum[3];
    __syncthreads();
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int r2 = min(r0 + rows_per_wg, a.N);
    int before = base;
    for (int r1 = r0; r1 < r2; r1 += 64) {
        const int mine = r1 + lane;
        const bool ok = mine < r2 && has_target(a, mine);
        const uint64_t m = __ballot(ok);
        if (wave == 0 && mine < r2) {
            const int at = ok ? before + lanes_below(m) : -1;
            a.ws.place[mine] = at;
            if (ok) {
                a.ws.target[at] = a.targets[mine];
                a.ws.source[at] = mine;
                if (a.grad_loss) {
                    a.ws.gscale[at] = a.scale * a.grad_loss[mine];
                    a.ws.lse[at] = a.lse_in[mine];
                }
            }
        }
        int k = 0;
        for (uint64_t rest = m; rest; rest &= rest - 1, ++k) {
            if ((k & 3) != wave) continue;
            const T* src = (const T*)a.hidden + (int64_t)(r1 + __builtin_ctzll(rest)) * a.hstride;
            const int64_t at = (int64_t)(before + k) * a.plan.Dp, plane = rows_cap * a.plan.Dp;
            if (what & kPackPlanes) pack_row(src, a.D, a.plan.Dp, a.ws.H + at, plane, lane, 64);
            if constexpr (sizeof(T) == 4) {
                if (what & kPackHalves) {
                    const float f = pack_row_half(src, a.D, a.plan.Dp, a.ws.Hh + at, plane, lane);
                    if (lane == 0) a.ws.hdown[before + k] = f;
                }
            }
        }
        if (zero_rows) {  // rows of grad_hidden without a target
            uint64_t none = ~m;
            if (r2 - r1 < 64) none &= (1ull << (r2 - r1)) - 1;
            for (k = 0; none; none &= none - 1, ++k) {
                if ((k & 3) != wave) continue;
                T* o = (T*)a.ghidden + (int64_t)(r1 + __builtin_ctzll(none)) * a.ghstride;
                for (int d = lane; d < a.D; d += 64) store_elem(o, d, 0.0f);
            }
        }
        before += __popcll(m);
    }
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) *a.ws.count = before;
}

// Words [v0, v0 + nv) of the table.
template <typename T>
__global__ __launch_bounds__(256) void pack_words_kernel(HeadArgs a, int v0, int nv, int what) {
    const int v = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (v >= nv) return;
    const T* src = (const T*)a.weight + (int64_t)(v0 + v) * a.wstride;
    const int64_t at = (int64_t)v * a.plan.Dp, plane = (int64_t)a.plan.Vw * a.plan.Dp;
    if (what & kPackPlanes) pack_row(src, a.D, a.plan.Dp, a.ws.W + at, plane, lane, 64);
    if constexpr (sizeof(T) == 4) {
        if (what & kPackHalves) {
            const float f = pack_row_half(src, a.D, a.plan.Dp, a.ws.Wh + at, plane, lane);
            if (lane == 0) a.ws.wdown[v] = f;
        }
    }
}

// ----------------------------------------------------------- tile order

__host__ __device__ inline int tiles_of(int64_t x, int t) { return (int)((x + t - 1) / t); }

// Workgroup b of tm x tn tiles: workgroups b, b + 8, ... run on one XCD (its own
// L2), so each XCD takes a contiguous run of tiles, in groups of 8 tile rows
// whose columns follow one another.
__device__ __forceinline__ void tile_of(int b, int tm, int tn, int& im, int& in) {
    const int total = tm * tn, q = total / 8, rem = total % 8, x = b % 8;
    const int id = x * q + (x < rem ? x : rem) + b / 8;
    const int per = 8 * tn, g = id / per, first = g * 8;
    const int gm = tm - first < 8 ? tm - first : 8;
    im = first + (id % per) % gm;
    in = (id % per) / gm;
}

// Shapes of the tiles by element type: large ones reuse each operand most; small
// ones fill the chip where there are few large ones, two to a CU or, where there
// is one to a CU at most, with more stages (deep): alone, a workgroup has only
// its own loads in flight to hide their latency.
enum Shape { kLarge, kSmall, kDeep };

template <typename T, bool AAcross, bool BAcross, Shape S>
struct TileFor;
template <bool AAcross, bool BAcross>
struct TileFor<uint16_t, AAcross, BAcross, kLarge> {
    typedef GemmTile<256, 256, 128, 64, 64, 1, AAcross, BAcross> type;
};
template <bool AAcross, bool BAcross>
struct TileFor<uint16_t, AAcross, BAcross, kSmall> {
    typedef GemmTile<128, 128, 64, 64, 64, 1, AAcross, BAcross> type;
};
template <bool AAcross, bool BAcross>
struct TileFor<uint16_t, AAcross, BAcross, kDeep> {
    typedef GemmTile<128, 128, 64, 64, 64, 1, AAcross, BAcross, false, 4> type;
};
template <bool AAcross, bool BAcross>
struct TileFor<float, AAcross, BAcross, kLarge> {
    typedef GemmTile<256, 128, 64, 64, 32, 3, AAcross, BAcross> type;
};
// three planes of a small tile's two stages leave a CU to one workgroup anyway
template <bool AAcross, bool BAcross>
struct TileFor<float, AAcross, BAcross, kSmall> {
    typedef GemmTile<128, 128, 64, 64, 32, 3, AAcross, BAcross, false, 3> type;
};
template <bool AAcross, bool BAcross>
struct TileFor<float, AAcross, BAcross, kDeep> : TileFor<float, AAcross, BAcross, kSmall> {};

// The logits' product: halves where the elements are fp32.
template <typename T, Shape S>
struct LogitTile {
    typedef typename TileFor<T, false, false, S>::type type;
};
template <>
struct LogitTile<float, kLarge> {
    typedef GemmTile<256, 256, 128, 64, 32, 2, false, false, true> type;
};
template <>
struct LogitTile<float, kSmall> {
    typedef GemmTile<128, 128, 64, 64, 32, 2, false, false, true> type;
};
template <>
struct LogitTile<float, kDeep> {
    typedef GemmTile<128, 128, 64, 64, 32, 2, false, false, true, 4> type;
};

template <typename Tile>
__device__ __forceinline__ Operand logit_hidden(const HeadArgs& a, int64_t rows_cap, int count) {
    return Operand{Tile::Half ? a.ws.Hh : a.ws.H, a.plan.Dp, rows_cap * a.plan.Dp, (int64_t)count * a.plan.Dp};
}
__device__ __forceinline__ Operand hidden_operand(const HeadArgs& a, int64_t rows_cap, int count) {
    return Operand{a.ws.H, a.plan.Dp, rows_cap * a.plan.Dp, (int64_t)count * a.plan.Dp};
}
__device__ __forceinline__ Operand grad_operand(const HeadArgs& a, int64_t rows_cap, int count) {
    return Operand{a.ws.G, a.plan.Vg, rows_cap * a.plan.Vg, (int64_t)count * a.plan.Vg};
}

// --------------------------------------------------- logits and their uses

constexpr int kPartWords = 64;  // of a part at least: sizes the parts' buffer

// Halves: the words' scales, divided out of a wave's accumulators (rows rm on of
// the piece); the hidden states' are left to their factors.
template <typename Tile>
__device__ __forceinline__ void unscale_words(const HeadArgs& a, int rm, f32x4v (&acc)[Tile::FM][Tile::FN]) {
    if (!Tile::Half) return;
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i) {
        const f32x4v w = *(const f32x4v*)(a.ws.wdown + rm + (i >> 1) * 32 + ((threadIdx.x & 63) >> 4) * 8 + (i & 1) * 4);
#pragma unroll
        for (int j = 0; j < Tile::FN; ++j) acc[i][j] *= w;
    }
}

// The loss's product.  Bound by the matrix cores: 7,370 packed rows of 2,048 bf16
// against 151,936 words take 3.6 ms, 1,270 TFLOP/s (torch's plain product of
// that size 1,370); fp32, 3,690 rows of 512 against 50,257 words: 0.5 ms, three
// 16-bit products at 1,130 TFLOP/s.  Words are the tile's rows so that a lane
// holds many words of one hidden state: a row's maximum and sum take two lane
// moves.  With 512 wide rows a tile has eight k steps, and its first loads and
// epilogue take as long as they.
//
// A wave's accumulators (gemm_tile.h): fragments 2i and 2i+1 of a lane hold the
// eight words rm + 32*i + (lane/16)*8 + 0..7 of hidden state rn + 16*j + lane%16.

template <typename Tile>
__global__ __launch_bounds__(Tile::NT) void head_parts_kernel(HeadArgs a, Operand W, int64_t rows_cap, int vp, int nv) {
    static_assert(Tile::WM >= kPartWords, "a part for each wave's words");
    __shared__ __align__(1024) char lds[Tile::Lds];
    const int count = *a.ws.count;
    int im, in;
    tile_of(blockIdx.x, tiles_of(nv, Tile::BM), tiles_of(a.N, Tile::BN), im, in);
    const int m0 = im * Tile::BM, n0 = in * Tile::BN;
    if (n0 >= count) return;
    f32x4v acc[Tile::FM][Tile::FN] = {};
    Tile::run(W, m0, logit_hidden<Tile>(a, rows_cap, count), n0, 0, a.D, lds, acc);

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int rm = m0 + (wave / (Tile::BN / Tile::WN)) * Tile::WM, rn = n0 + (wave % (Tile::BN / Tile::WN)) * Tile::WN;
    if (rm >= nv) return;
    const int vl = vp + rm + (lane >> 4) * 8;  // word of acc[0][j][0]
    const int part = (vp + rm) / Tile::WM;
    unscale_words<Tile>(a, rm, acc);
    float down[Tile::FN];  // the row's factor: the logits' scale, and its own
#pragma unroll
    for (int j = 0; j < Tile::FN; ++j) {
        const int n = rn + j * 16 + (lane & 15);
        down[j] = Tile::Half && n < count ? a.scale * a.ws.hdown[n] : a.scale;
        const int t = n < count ? a.ws.target[n] - vl : -1;
        if (__ballot(t >= 0 && t < Tile::WM) == 0) continue;
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if ((i >> 1) * 32 + (i & 1) * 4 + r == t) a.ws.zt[n] = acc[i][j][r] * down[j];
    }
    // from here on in units of log 2: y = z log2 e
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i)
#pragma unroll
        for (int j = 0; j < Tile::FN; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][j][r] *= down[j] * kLog2e;
    if (vp + rm + Tile::WM > a.V) {  // words behind the table take no part
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (vl + (i >> 1) * 32 + (i & 1) * 4 + r >= a.V)
#pragma unroll
                    for (int j = 0; j < Tile::FN; ++j) acc[i][j][r] = kFarBelow;
    }
#pragma unroll
    for (int j = 0; j < Tile::FN; ++j) {
        const int n = rn + j * 16 + (lane & 15);
        float m = kFarBelow;
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) m = fmaxf(m, acc[i][j][r]);
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) s += ex2(acc[i][j][r] - m);
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (lane < 16 && n < count) a.ws.parts[(int64_t)part * rows_cap + n] = make_float2(m, s);
    }
}

// The normaliser from a row's maximum and sum in units of log 2.
__device__ __forceinline__ float lse_of(float m, float s) { return (float)(kLn2 * ((double)m + (double)log2f(s))); }

// Loss and lse of each row from its parts: workgroups of `rb` rows, 1024 / rb
// threads to a row.  packed: the rows are pack_rows_kernel's.
__global__ __launch_bounds__(1024) void head_join_kernel(HeadArgs a, int64_t rows_cap, int parts, int rb, bool packed) {
    __shared__ float sm[1024], ss[1024];
    const int slices = 1024 / rb, row = threadIdx.x % rb, slice = threadIdx.x / rb;
    const int n = blockIdx.x * rb + row;
    const int at = n >= a.N ? -1 : packed ? a.ws.place[n] : has_target(a, n) ? n : -1;
    float m = kFarBelow, s = 0.0f;
    if (at >= 0)
        for (int p = slice; p < parts; p += slices) {
            const float2 x = a.ws.parts[(int64_t)p * rows_cap + at];
            const float hi = fmaxf(m, x.x);
            s = s * ex2(m - hi) + x.y * ex2(x.x - hi);
            m = hi;
        }
    sm[threadIdx.x] = m;
    ss[threadIdx.x] = s;
    for (int half = slices / 2; half; half >>= 1) {
        __syncthreads();
        if (slice < half) {
            const int o = threadIdx.x + half * rb;
            const float hi = fmaxf(sm[threadIdx.x], sm[o]);
            ss[threadIdx.x] = ss[threadIdx.x] * ex2(sm[threadIdx.x] - hi) + ss[o] * ex2(sm[o] - hi);
            sm[threadIdx.x] = hi;
        }
    }
    if (slice == 0 && n < a.N) {
        float lse = 0.0f, loss = 0.0f;
        if (at >= 0) {
            lse = lse_of(sm[row], ss[row]);
            loss = lse - a.ws.zt[at];
        }
        a.loss[n] = loss;
        a.lse[n] = lse;
    }
}

// ------------------------------------------------------------- few rows

// Forward of at most 64 rows: bound by reading the table once.  A workgroup
// takes 16 words a wave; the words go from memory straight to the matrix cores'
// registers (two k steps ahead), fp32 ones split into planes on the way, since
// each is used by one wave only.  The hidden states, which every wave needs, go
// through LDS a k step at a time.  Nothing is packed before: rows without a
// target are staged as zeros.  One row of 2,048 bf16 against 151,936 words: 111
// us, 5.6 TB/s of the 6.9 that a plain read reaches; 64 rows of 768 fp32 against
// 50,257 words: 41 us, where LDS reads, matrix and vector instructions of a
// step are each a third.
constexpr int kFewRows = 64;

template <typename T>
struct Raw8;  // eight elements as loaded
template <>
struct Raw8<uint16_t> {
    u32x4 v;
    __device__ __forceinline__ void load(const uint16_t* p, int d, int D) { v = load8_bits(p, d, D); }
    __device__ __forceinline__ void zero() { v = u32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ void planes(bf16x8 (&b)[1]) const { b[0] = __builtin_bit_cast(bf16x8, v); }
};
template <>
struct Raw8<float> {
    float x[8];
    __device__ __forceinline__ void load(const float* p, int d, int D) { load8(p, d, D, x); }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.0f;
    }
    __device__ __forceinline__ void planes(bf16x8 (&b)[3]) const {
        u32x4 t[3];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t h[3];
            split_pair<3>(x[2 * e], x[2 * e + 1], h);
#pragma unroll
            for (int p = 0; p < 3; ++p) t[p][e] = h[p];
        }
#pragma unroll
        for (int p = 0; p < 3; ++p) b[p] = __builtin_bit_cast(bf16x8, t[p]);
    }
};

template <typename T, int FN, int MinWaves, int MaxWaves, int StepK>
__global__ __launch_bounds__(MaxWaves * 64) void head_stream_kernel(HeadArgs a) {
    static_assert(MinWaves * 16 >= kPartWords, "a part for each workgroup");
    const int NT = blockDim.x, waves = NT / 64;  // MinWaves .. MaxWaves
    constexpr int PL = sizeof(T) == 2 ? 1 : 3, kRows = FN * 16, kChunks = StepK / 8;
    constexpr int kItems = (kRows * kChunks + MinWaves * 64 - 1) / (MinWaves * 64), kParts32 = StepK / 32;
    __shared__ __align__(16) uint16_t hs[2][PL][kRows][StepK];
    __shared__ float sm[MaxWaves][kRows], ss[MaxWaves][kRows], szt[kRows];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int v0 = (blockIdx.x * waves + wave) * 16;
    const int steps = tiles_of(a.D, StepK);
    // the width is walked in a circle from another step in every workgroup: rows
    // of the table lie a power of two apart as often as not, and workgroups in
    // step with one another would all ask the same memory channels
    const int turn = (int)(blockIdx.x * 5u % (unsigned)steps);

    // this thread's 16-byte chunks of the hidden states' step
    const T* hrow[kItems];
    bool hok[kItems];
#pragma unroll
    for (int q = 0; q < kItems; ++q) {
        const int n = (q * NT + threadIdx.x) / kChunks;
        hok[q] = n < kRows && has_target(a, n);
        hrow[q] = (const T*)a.hidden + (int64_t)(hok[q] ? n : 0) * a.hstride;
    }
    Raw8<T> hr[kItems];
    const auto fetch_h = [&](int c) {
        c += turn;
        c -= c >= steps ? steps : 0;
#pragma unroll
        for (int q = 0; q < kItems; ++q) {
            const int d = c * StepK + (threadIdx.x % kChunks) * 8;
            if (hok[q] && d < a.D) hr[q].load(hrow[q], d, a.D);
            else hr[q].zero();
        }
    };
    const auto stage_h = [&](int buf) {
#pragma unroll
        for (int q = 0; q < kItems; ++q) {
            const int n = (q * NT + threadIdx.x) / kChunks;
            if (n >= kRows) continue;
            bf16x8 b[PL];
            hr[q].planes(b);
#pragma unroll
            for (int p = 0; p < PL; ++p)
                *(bf16x8*)&hs[buf][p][n][((threadIdx.x % kChunks) ^ along_swz<8, false>(n)) * 8] = b[p];
        }
    };
    const T* wrow = (const T*)a.weight + (int64_t)min(a.V - 1, v0 + (lane & 15)) * a.wstride;
    struct Words {
        Raw8<T> r[kParts32];
    } w0, w1;
    const auto fetch_w = [&](Words& w, int c) {
        c += turn;
        c -= c >= steps ? steps : 0;
#pragma unroll
        for (int kk = 0; kk < kParts32; ++kk) {
            const int d = c * StepK + kk * 32 + (lane >> 4) * 8;
            if (d < a.D) w.r[kk].load(wrow, d, a.D);
            else w.r[kk].zero();
        }
    };
    f32x4v acc[FN] = {};
    const auto step = [&](int c, Words& w) {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's LDS writes and reads
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (c + 1 < steps) stage_h((c + 1) & 1);
        if (c + 2 < steps) fetch_h(c + 2);
#pragma unroll
        for (int kk = 0; kk < kParts32; ++kk) {
            bf16x8 b[PL][FN];
#pragma unroll
            for (int p = 0; p < PL; ++p)
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    const int n = j * 16 + (lane & 15);
                    b[p][j] = *(const bf16x8*)&hs[c & 1][p][n][((kk * 4 + (lane >> 4)) ^ along_swz<8, false>(n)) * 8];
                }
            bf16x8 x[PL];
            w.r[kk].planes(x);
#pragma unroll
            for (int sum = PL - 1; sum >= 0; --sum)
#pragma unroll
                for (int pa = sum; pa >= 0; --pa)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[pa], b[sum - pa][j], acc[j], 0, 0, 0);
        }
        if (c + 2 < steps) fetch_w(w, c + 2);
    };
    fetch_w(w0, 0);
    fetch_h(0);
    stage_h(0);
    if (steps > 1) {
        fetch_h(1);
        fetch_w(w1, 1);
    }
    for (int c = 0; c < steps; c += 2) {
        step(c, w0);
        if (c + 1 < steps) step(c + 1, w1);
    }

#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const int n = j * 16 + (lane & 15);
        const int t = has_target(a, n) ? a.targets[n] - v0 - (lane >> 4) * 4 : -1;
        float m = kFarBelow, s = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (t == r) szt[n] = acc[j][r] * a.scale;  // at most one lane of the workgroup
            acc[j][r] *= a.scale * kLog2e;
            if (v0 + (lane >> 4) * 4 + r < a.V) m = fmaxf(m, acc[j][r]);
        }
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (v0 + (lane >> 4) * 4 + r < a.V) s += ex2(acc[j][r] - m);
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (lane < 16) {
            sm[wave][n] = m;
            ss[wave][n] = s;
        }
    }
    __syncthreads();
    if ((int)threadIdx.x < kRows && (int)threadIdx.x < a.N) {
        const int n = threadIdx.x;
        float m = sm[0][n], s = 0.0f;
        for (int w = 1; w < waves; ++w) m = fmaxf(m, sm[w][n]);
        for (int w = 0; w < waves; ++w) s += ss[w][n] * ex2(sm[w][n] - m);
        const int t = has_target(a, n) ? a.targets[n] : -1;
        if (gridDim.x == 1) {  // the whole vocabulary: nothing to join
            const float lse = t < 0 ? 0.0f : lse_of(m, s);
            a.lse[n] = lse;
            a.loss[n] = t < 0 ? 0.0f : lse - szt[n];
            return;
        }
        a.ws.parts[(int64_t)blockIdx.x * a.N + n] = make_float2(m, s);
        if (t >= 0 && t / (waves * 16) == (int)blockIdx.x) a.ws.zt[n] = szt[n];
    }
}

// A piece's G.  bf16: rounded to nearest, an error of half a step of each
// element where the products' sums are of thousands; fp32: three planes.  The
// loss's product again with another epilogue: 0.80 ms for 30,464 words of the
// bf16 case there, 1,150 TFLOP/s, 450 MB of G written.
template <typename Tile>
__global__ __launch_bounds__(Tile::NT) void head_grad_kernel(HeadArgs a, Operand W, int64_t rows_cap, int vp, int nv) {
    __shared__ __align__(1024) char lds[Tile::Lds];
    constexpr int PL = Tile::Half ? 3 : Tile::PL;  // of G
    const int count = *a.ws.count;
    int im, in;
    tile_of(blockIdx.x, tiles_of(nv, Tile::BM), tiles_of(a.N, Tile::BN), im, in);
    const int m0 = im * Tile::BM, n0 = in * Tile::BN;
    if (n0 >= count) return;
    f32x4v acc[Tile::FM][Tile::FN] = {};
    Tile::run(W, m0, logit_hidden<Tile>(a, rows_cap, count), n0, 0, a.D, lds, acc);

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int rm = m0 + (wave / (Tile::BN / Tile::WN)) * Tile::WM, rn = n0 + (wave % (Tile::BN / Tile::WN)) * Tile::WN;
    const int vl = rm + (lane >> 4) * 8;
    const int64_t plane = rows_cap * a.plan.Vg;
    const bool whole = rm + Tile::WM <= nv;
    unscale_words<Tile>(a, rm, acc);
#pragma unroll
    for (int j = 0; j < Tile::FN; ++j) {
        const int n = rn + j * 16 + (lane & 15);
        if (n >= count) continue;
        const int t = a.ws.target[n] - vp - vl;
        const float g = a.ws.gscale[n], lse = a.ws.lse[n], lse2 = lse * kLog2e;
        const bool hit = __ballot(t >= 0 && t < Tile::WM) != 0;
        const float down = Tile::Half ? a.scale * a.ws.hdown[n] : a.scale, c = down * kLog2e;
#pragma unroll
        for (int i = 0; i < Tile::FM; i += 2) {
            u32x4 out[PL];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                float x[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int o = (i >> 1) * 32 + e + q;
                    // fp32: the difference first, or the roundings of the two
                    // terms stay in a probability near one
                    const float z = acc[i + (e >> 2)][j][(e & 3) + q];
                    float p = PL == 1 ? ex2(fmaf(z, c, -lse2)) : ex2(fmaf(z, down, -lse) * kLog2e);
                    if (hit && o == t) p -= 1.0f;
                    x[q] = whole || vl + o < nv ? g * p : 0.0f;
                }
                uint32_t b[PL];
                split_pair<PL>(x[0], x[1], b);
#pragma unroll
                for (int pl = 0; pl < PL; ++pl) out[pl][e >> 1] = b[pl];
            }
            // the buffer's rows hold whole tiles: words behind the piece are zero
            uint16_t* dst = a.ws.G + (int64_t)n * a.plan.Vg + vl + (i >> 1) * 32;
#pragma unroll
            for (int pl = 0; pl < PL; ++pl) *(u32x4*)(dst + pl * plane) = out[pl];
        }
    }
}

// ------------------------------------------------------------- gradients

// Four elements of a row of an output, 8 or 16 bytes at once; `add`: to what it
// holds; only `left` of them exist.
__device__ __forceinline__ void put4(float* o, int left, bool add, f32x4v x) {
    if (left >= 4) {
        if (add) x += *(const f32x4_anywhere*)o;
        *(f32x4_anywhere*)o = x;
        return;
    }
    for (int r = 0; r < 4; ++r)
        if (r < left) o[r] = add ? o[r] + x[r] : x[r];
}
__device__ __forceinline__ void put4(uint16_t* o, int left, bool add, f32x4v x) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    typedef u32x2 Anywhere __attribute__((aligned(2)));
    if (left >= 4) {
        if (add) {
            const u32x2 old = *(const Anywhere*)o;
            x += f32x4v{__uint_as_float(old[0] << 16), __uint_as_float(old[0] & 0xFFFF0000u), __uint_as_float(old[1] << 16),
                        __uint_as_float(old[1] & 0xFFFF0000u)};
        }
        *(Anywhere*)o = u32x2{bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3])};
        return;
    }
    for (int r = 0; r < 4; ++r)
        if (r < left) o[r] = bf16_bits(add ? bf16_value(o[r]) + x[r] : x[r]);
}
// Split s of the piece's words: its share of grad_hidden, added to what the
// pieces before left.  out: the last piece of an unsplit product writes the
// rows themselves (an own pass over the fp32 sums took 33 us more for 40,960
// rows of 512).  0.82 ms for the piece above, 1,120 TFLOP/s: a tenth of the
// tiles are behind the packed rows, whose number the host does not know.
template <typename T, typename Tile>
__global__ __launch_bounds__(Tile::NT) void head_ghidden_kernel(HeadArgs a, Operand W, int64_t rows_cap, int nv, int splits,
                                                                bool first, bool out) {
    __shared__ __align__(1024) char lds[Tile::Lds];
    const int count = *a.ws.count;
    const int tm = tiles_of(a.D, Tile::BM), tn = tiles_of(a.N, Tile::BN);
    const int s = blockIdx.x / (tm * tn);
    int im, in;
    tile_of(blockIdx.x % (tm * tn), tm, tn, im, in);
    const int m0 = im * Tile::BM, n0 = in * Tile::BN;
    if (n0 >= count) return;
    const int per = tiles_of(tiles_of(nv, Tile::BK), splits) * Tile::BK;
    const int k0 = s * per, k1 = min(nv, k0 + per);
    f32x4v acc[Tile::FM][Tile::FN] = {};
    // k behind the piece: G's words there are zero up to its row's end
    Tile::run(W, m0, grad_operand(a, rows_cap, count), n0, k0, k1, lds, acc);

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int rm = m0 + (wave / (Tile::BN / Tile::WN)) * Tile::WM, rn = n0 + (wave % (Tile::BN / Tile::WN)) * Tile::WN;
    float* gh = a.ws.gh + (int64_t)s * a.N * a.plan.Dp;
#pragma unroll
    for (int j = 0; j < Tile::FN; ++j) {
        const int n = rn + j * 16 + (lane & 15);
        if (n >= count) continue;
        T* row = out ? (T*)a.ghidden + (int64_t)a.ws.source[n] * a.ghstride : nullptr;
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) {
            const int d = rm + i * 16 + (lane >> 4) * 4;
            if (d >= a.plan.Dp) continue;
            f32x4v* o = (f32x4v*)(gh + (int64_t)n * a.plan.Dp + d);
            const f32x4v x = first ? acc[i][j] : *o + acc[i][j];
            if (out) put4(row + d, a.D - d, false, x);
            else *o = x;
        }
    }
}

// grad_hidden of a split product: the splits' sums in order, one rounding; zero
// without a target.
template <typename T>
__global__ __launch_bounds__(256) void head_ghidden_out_kernel(HeadArgs a, int splits) {
    const int n = blockIdx.x;
    const int at = a.ws.place[n];
    const int64_t stride = (int64_t)a.N * a.plan.Dp;
    for (int d = threadIdx.x * 4; d < a.D; d += 1024) {
        f32x4v s = {};
        if (at >= 0)
#pragma unroll 8
            for (int q = 0; q < splits; ++q) s += *(const f32x4v*)(a.ws.gh + q * stride + (int64_t)at * a.plan.Dp + d);
        put4((T*)a.ghidden + (int64_t)n * a.ghstride + d, a.D - d, false, s);
    }
}

// The piece's rows of grad_weight, or (splits > 1) partial sums of them over a
// split of the packed rows: 1,280 words of 512 have ten tiles, 25 splits of
// 40,960 rows fill the chip (66 us against 118 in small tiles).  0.80 ms for the
// piece above, 1,150 TFLOP/s.
template <typename T, typename Tile>
__global__ __launch_bounds__(Tile::NT) void head_gweight_kernel(HeadArgs a, int64_t rows_cap, int vp, int nv, int splits) {
    __shared__ __align__(1024) char lds[Tile::Lds];
    const int count = *a.ws.count;
    const int tm = tiles_of(a.D, Tile::BM), tn = tiles_of(nv, Tile::BN);
    const int s = blockIdx.x / (tm * tn);
    int im, in;
    tile_of(blockIdx.x % (tm * tn), tm, tn, im, in);
    const int m0 = im * Tile::BM, n0 = in * Tile::BN;
    const int per = tiles_of(tiles_of(count, Tile::BK), splits) * Tile::BK;
    const int k0 = s * per, k1 = min(count, k0 + per);
    f32x4v acc[Tile::FM][Tile::FN] = {};
    Tile::run(hidden_operand(a, rows_cap, count), m0, grad_operand(a, rows_cap, count), n0, k0, k1, lds, acc);

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int rm = m0 + (wave / (Tile::BN / Tile::WN)) * Tile::WM, rn = n0 + (wave % (Tile::BN / Tile::WN)) * Tile::WN;
#pragma unroll
    for (int j = 0; j < Tile::FN; ++j) {
        const int v = rn + j * 16 + (lane & 15);
        if (v >= nv) continue;
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) {
            const int d = rm + i * 16 + (lane >> 4) * 4;
            if (d >= a.plan.Dp) continue;
            if (splits > 1) *(f32x4v*)(a.ws.gw + ((int64_t)s * nv + v) * a.plan.Dp + d) = acc[i][j];
            else put4((T*)a.gweight + (int64_t)(vp + v) * a.gwstride + d, a.D - d, a.accumulate, acc[i][j]);
        }
    }
}

template <typename T>
__global__ __launch_bounds__(256) void head_gweight_out_kernel(HeadArgs a, int vp, int nv, int splits) {
    const int v = blockIdx.x;
    for (int d = threadIdx.x * 4; d < a.D; d += 1024) {
        f32x4v s = {};
#pragma unroll 8
        for (int q = 0; q < splits; ++q) s += *(const f32x4v*)(a.ws.gw + ((int64_t)q * nv + v) * a.plan.Dp + d);
        put4((T*)a.gweight + (int64_t)(vp + v) * a.gwstride + d, a.D - d, a.accumulate, s);
    }
}

template <typename T>
__global__ __launch_bounds__(256) void head_zero_kernel(HeadArgs a) {
    for (int d = threadIdx.x; d < a.D; d += 256) store_elem((T*)a.gweight + (int64_t)blockIdx.x * a.gwstride, d, 0.0f);
}

// ------------------------------------------------------------ small problems

// The loss, or the whole backward, in one launch, where several would cost more
// than the work.  Backward: a workgroup takes 16 rows of grad_hidden or 16 rows of
// grad_weight, computes the slab of G it needs (so each logit is computed twice)
// into LDS in fp32 and multiplies it.  fp32 matrix instructions throughout, bf16
// elements widened; no rounding of G.  48 rows, 48 words, 64 wide: 5.2 us, a chain
// of loads.  A k of four is spread over a lane's four consecutive elements: both
// operands agree on which.
constexpr int kSmallMost = 512;  // rows and words at most: their share of G is 33 KB of LDS

__device__ __forceinline__ f32x4v load4(const float* p) { return *(const f32x4_anywhere*)p; }
__device__ __forceinline__ f32x4v load4(const uint16_t* p) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    typedef u32x2 Anywhere __attribute__((aligned(2)));
    const u32x2 v = *(const Anywhere*)p;
    return f32x4v{__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xFFFF0000u), __uint_as_float(v[1] << 16),
                  __uint_as_float(v[1] & 0xFFFF0000u)};
}

// The logits (unscaled) of 16 words and 16 hidden states, each lane giving its
// lane%16-th word v and state n: a lane gets words 4*(lane/16) .. +3 of its state,
// zero where either is not in.  Loads are from clamped places and unconditional (a
// branch around each would leave one in flight); what is not in is zeroed behind them.
template <typename T>
__device__ __forceinline__ f32x4v small_logits(const HeadArgs& a, int v, bool vin, int n, bool nin) {
    const int lk = (threadIdx.x & 63) >> 4;
    const T* wp = (const T*)a.weight + (int64_t)(vin ? v : 0) * a.wstride;
    const T* hp = (const T*)a.hidden + (int64_t)(nin ? n : 0) * a.hstride;
    f32x4v acc = {};
    int d0 = 0;
#pragma unroll 4
    for (; d0 + 16 <= a.D; d0 += 16) {
        const f32x4v x = load4(wp + d0 + lk * 4), y = load4(hp + d0 + lk * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(vin ? x[e] : 0.0f, nin ? y[e] : 0.0f, acc, 0, 0, 0);
    }
    for (; d0 < a.D; d0 += 16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int d = d0 + lk * 4 + e, at = min(d, a.D - 1);
            const float x = load_elem(wp, at), y = load_elem(hp, at);
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(vin && d < a.D ? x : 0.0f, nin && d < a.D ? y : 0.0f, acc, 0, 0, 0);
        }
    }
    return acc;
}

// The loss of a small problem: 16 rows to a workgroup, 16 threads to a row.  48
// rows, 48 words, 64 wide: 4.1 us.  The backward below makes the same logits to
// the bit, which leaves a probability near one as near to it: gradients of those
// sizes are 3e-7 of their norm off where a loss by other sums left 1.1e-6.
template <typename T>
__global__ __launch_bounds__(256) void head_small_loss_kernel(HeadArgs a) {
    extern __shared__ __align__(16) float zs[];  // [16][pitch]: rows x words
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, li = lane & 15, lk = lane >> 4;
    const int r0 = blockIdx.x * 16, pitch = (a.V + 15) / 16 * 16 + 4;
    const bool nin = has_target(a, r0 + li);
    for (int v0 = wave * 16; v0 < a.V; v0 += 64) {
        const f32x4v acc = small_logits<T>(a, v0 + li, v0 + li < a.V, r0 + li, nin);
#pragma unroll
        for (int r = 0; r < 4; ++r) zs[li * pitch + v0 + lk * 4 + r] = acc[r] * a.scale;
    }
    __syncthreads();
    const int row = threadIdx.x >> 4, c = threadIdx.x & 15, n = r0 + row;
    const float* z = zs + row * pitch;
    float m = kFarBelow, s = 0.0f;
    for (int v = c; v < a.V; v += 16) m = fmaxf(m, z[v] * kLog2e);
#pragma unroll
    for (int o = 1; o < 16; o *= 2) m = fmaxf(m, __shfl_xor(m, o));
    for (int v = c; v < a.V; v += 16) s += ex2(z[v] * kLog2e - m);
#pragma unroll
    for (int o = 1; o < 16; o *= 2) s += __shfl_xor(s, o);
    if (c == 0 && n < a.N) {
        const bool ok = has_target(a, n);
        const float lse = ok ? lse_of(m, s) : 0.0f;
        a.lse[n] = lse;
        a.loss[n] = ok ? lse - z[a.targets[n]] : 0.0f;
    }
}

template <typename T>
__global__ __launch_bounds__(256) void head_small_backward_kernel(HeadArgs a, int row_wgs) {
    extern __shared__ __align__(16) float gs[];  // [16][pitch]: rows (or words) x words (or rows)
    __shared__ bool there[kSmallMost];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, li = lane & 15, lk = lane >> 4;
    const bool rows = (int)blockIdx.x < row_wgs;  // grad_hidden's workgroup
    const int r0 = rows ? blockIdx.x * 16 : 0, w0 = rows ? 0 : (blockIdx.x - row_wgs) * 16;
    const int others = rows ? a.V : a.N;  // the length of the second product
    const int pitch = (others + 15) / 16 * 16 + 4;

    for (int o0 = wave * 16; o0 < others; o0 += 64) {
        const int v = (rows ? o0 : w0) + li, n = (rows ? r0 : o0) + li;
        const bool vin = v < a.V, nin = has_target(a, n);
        const float g = nin ? a.scale * a.grad_loss[n] : 0.0f, lse = nin ? a.lse_in[n] : 0.0f;
        const int t = nin ? a.targets[n] - (v - li) : -1;
        const f32x4v acc = small_logits<T>(a, v, vin, n, nin);
        // acc[r]: word 4*lk + r of the tile, row li
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int w = lk * 4 + r;
            float p = ex2(fmaf(acc[r], a.scale, -lse) * kLog2e);
            if (w == t) p -= 1.0f;
            const float x = nin && v - li + w < a.V ? g * p : 0.0f;
            if (rows) gs[li * pitch + o0 + w] = x;
            else gs[w * pitch + o0 + li] = x;
        }
        // which rows of the second product's left side exist
        if (lk == 0) there[o0 + li] = rows ? vin : nin;
    }
    __syncthreads();
    const int mine = (rows ? r0 : w0) + li;  // this lane's row of the output
    const bool stored = mine < (rows ? a.N : a.V);
    const bool zero = rows && !has_target(a, mine);
    T* out = rows ? (T*)a.ghidden + (int64_t)mine * a.ghstride : (T*)a.gweight + (int64_t)mine * a.gwstride;
    const T* left = rows ? (const T*)a.weight : (const T*)a.hidden;
    const int64_t lstride = rows ? a.wstride : a.hstride;
    const int padded = (others + 15) / 16 * 16;
    for (int d0 = wave * 16; d0 < a.D; d0 += 64) {
        f32x4v acc = {};
        const T* col = left + min(d0 + li, a.D - 1);
#pragma unroll 2
        for (int k0 = 0; k0 < padded; k0 += 16) {
#pragma unroll
            for (int q = 0; q < 16; q += 4) {
                const int k = k0 + q + lk;
                const float x = load_elem(col, (int64_t)min(k, others - 1) * lstride);
                acc = __builtin_amdgcn_mfma_f32_16x16x4f32(there[k] ? x : 0.0f, gs[li * pitch + k], acc, 0, 0, 0);
            }
        }
        const int od = d0 + lk * 4;
        if (stored && od < a.D) put4(out + od, a.D - od, !rows && a.accumulate, zero ? f32x4v{} : acc);
    }
}

// ------------------------------------------------------------------ host

constexpr int kMaxSplits = 64;
constexpr int kCUs = 256;
constexpr int kLdsBytes = 160 << 10;  // of a CU

// How a product of m x n with k steps is cut: into tiles of a shape, the k axis
// into splits.  The cost is in k steps of a large tile: rounds of workgroups over
// the chip, each its k steps and `ends` more for its first loads and its
// epilogue; small tiles work at four fifths of the large ones' rate where two
// share a CU, at about half of it alone (one wave to a SIMD).  Splits pay
// for writing and reading their fp32 sums: a CU moves a large tile's in about
// six k steps, and the launch that adds them takes about two and a half.  Only
// splits that fill one, two or three rounds can be the best.
struct Cut {
    Shape shape;
    int splits;
    double cost;
};
constexpr int kMostRounds = 3;  // of a split product

template <typename Large, typename Tile>
void try_cut(Shape shape, int64_t m, int64_t n, int64_t k, bool may_split, double ends, Cut* best) {
    constexpr int kShare = 2 * Tile::Lds <= kLdsBytes ? 2 : 1;  // workgroups on a CU
    constexpr double kRate = Tile::BM * Tile::BN == Large::BM * Large::BN ? 1.0 : kShare == 2 ? 0.8 : 0.55;
    constexpr double kStep = (double)kShare * Tile::BM * Tile::BN * Tile::BK / (Large::BM * Large::BN * Large::BK) / kRate;
    const int64_t tiles = (int64_t)tiles_of(m, Tile::BM) * tiles_of(n, Tile::BN);
    const int steps = tiles_of(k, Tile::BK), slots = kShare * kCUs;
    if (shape == kDeep && tiles > slots) return;  // small tiles then, two to a CU
    for (int round = 0; round <= (may_split ? kMostRounds : 0); ++round) {
        int64_t s = 1;
        if (round > 0) {
            s = (int64_t)round * slots / tiles;
            if (s > kMaxSplits) s = kMaxSplits;
            if (s > steps / 4) s = steps / 4;  // four k steps each, or more
            if (s < 2) continue;
        }
        const double rounds = (double)((tiles * s + slots - 1) / slots);
        double cost = rounds * ((double)((steps + s - 1) / s) + ends) * kStep;
        if (s > 1) cost += 6.0 * kStep * (double)(tiles * s) / slots + 2.5;
        if (cost < best->cost * 0.999) *best = Cut{shape, (int)s, cost};
    }
}

template <typename Large, typename Small, typename Deep>
Cut cut_product(int64_t m, int64_t n, int64_t k, bool may_split, double ends) {
    Cut best{kLarge, 1, 1e300};
    try_cut<Large, Large>(kLarge, m, n, k, may_split, ends, &best);
    try_cut<Large, Small>(kSmall, m, n, k, may_split, ends, &best);
    try_cut<Large, Deep>(kDeep, m, n, k, may_split, ends, &best);
    return best;
}

constexpr double kLogitEnds = 7, kSumEnds = 4;  // of the logits and of the gradients

template <typename T>
Cut cut_logits(int64_t words, int64_t rows, int64_t dim) {
    return cut_product<typename LogitTile<T, kLarge>::type, typename LogitTile<T, kSmall>::type, typename LogitTile<T, kDeep>::type>(
        words, rows, dim, false, kLogitEnds);
}
template <typename T, bool BAcross>
Cut cut_gradient(int64_t m, int64_t n, int64_t k) {
    return cut_product<typename TileFor<T, true, BAcross, kLarge>::type, typename TileFor<T, true, BAcross, kSmall>::type,
                       typename TileFor<T, true, BAcross, kDeep>::type>(m, n, k, true, kSumEnds);
}

constexpr int64_t kPieceElems = 256ll << 20;   // of the logits' gradient at most (512 MB)
constexpr int64_t kTableElems = 128ll << 20;   // of a packed piece of the table, all planes
constexpr int64_t kPartRows = 65536;           // rows of a forward pass
constexpr int kWordTile = 256;                 // pieces are whole tiles of any shape

// Whether rows of 16-bit elements can be read as they lie: whole 16-byte
// chunks, and offsets within a tile that fit 32 bits.
bool reads_in_place(const void* p, int64_t stride, int D, int dtype) {
    return dtype == GR_BF16 && D % 8 == 0 && stride % 8 == 0 && stride <= kMaxTileStride && (uintptr_t)p % 16 == 0;
}

template <typename T>
hipError_t pack_rows(const HeadArgs& a, int64_t cap, int what, bool zero_rows, hipStream_t st) {
    // a row to a wave while there are few; the counts before the workgroups'
    // rows are quadratic in the workgroups' number
    int per = 4;
    while (tiles_of(a.N, per) > (per < 16 ? 2048 : 4096)) per *= 2;
    pack_rows_kernel<T><<<dim3((unsigned)tiles_of(a.N, per)), 256, 0, st>>>(a, cap, per, what, zero_rows);
    return hipGetLastError();
}

// Words [v, v + nv) as the operand of the logits and of grad_hidden, packed first
// where they cannot be read in place.
struct Words {
    Operand logits, planes;
};

template <typename T>
Words words_operands(const HeadArgs& a, int v, int nv, bool planes, int dtype, hipStream_t st) {
    const int Dp = a.plan.Dp;
    if (reads_in_place(a.weight, a.wstride, a.D, dtype)) {
        const uint16_t* p = (const uint16_t*)a.weight + (int64_t)v * a.wstride;
        const Operand w{p, a.wstride, 0, (int64_t)(nv - 1) * a.wstride + a.D};
        return Words{w, w};
    }
    const int64_t plane = (int64_t)a.plan.Vw * Dp;
    const bool half = sizeof(T) == 4;
    const int what = half ? kPackHalves + (planes ? kPackPlanes : 0) : kPackPlanes;
    pack_words_kernel<T><<<dim3((unsigned)tiles_of(nv, 4)), 256, 0, st>>>(a, v, nv, what);
    return Words{Operand{half ? a.ws.Wh : a.ws.W, Dp, plane, (int64_t)nv * Dp}, Operand{a.ws.W, Dp, plane, (int64_t)nv * Dp}};
}

template <typename Tile>
void run_parts(const HeadArgs& a, const Operand& W, int64_t cap, int v, int nv, hipStream_t st) {
    head_parts_kernel<Tile><<<dim3((unsigned)(tiles_of(nv, Tile::BM) * tiles_of(a.N, Tile::BN))), Tile::NT, 0, st>>>(a, W, cap, v, nv);
}

// One launch: at most one workgroup to a CU, and no longer a walk of each wave
// than the other way's launches cost.  A walk of 512: 4,096 fp32 rows of 512
// against 64 words 12 us against 33, 512 bf16 rows of 64 against 512 words 14
// against 16; of 2,000: 64 bf16 rows against 16 words 31 against 21, 64 fp32 rows
// of 256 against 512 words 36 against 18.  16,384 bf16 rows of 512 against 64
// words, four workgroups to a CU: 33 against 27.  Up to kFewRows rows the other way
// is two launches, and the walk 256: 8 bf16 rows of 64 against 512 words (a walk of
// 512), 3.7 and 4.2 us of kernels by it against 11.6.
bool small_loss(const HeadArgs& a) {
    return a.N <= 4096 && a.V <= kSmallMost && (int64_t)tiles_of(a.V, 64) * a.D <= (a.N <= kFewRows ? 256 : 512);
}

template <typename T>
hipError_t head_loss_t(const HeadArgs& all, int dtype, hipStream_t st) {
    const int64_t cap = all.plan.part_rows;
    if (small_loss(all)) {
        const size_t lds = 16 * (size_t)(tiles_of(all.V, 16) * 16 + 4) * sizeof(float);
        head_small_loss_kernel<T><<<dim3((unsigned)tiles_of(all.N, 16)), 256, lds, st>>>(all);
        return hipGetLastError();
    }
    for (int64_t r = 0; r < all.N; r += cap) {
        HeadArgs a = all;
        a.N = (int32_t)(all.N - r < cap ? all.N - r : cap);
        a.hidden = (const T*)all.hidden + r * all.hstride;
        a.targets = all.targets + r;
        a.loss = all.loss + r;
        a.lse = all.lse + r;
        a.grad_loss = nullptr;
        if (a.N <= kFewRows) {
            // More rows: more waves share the staging of the hidden states, which
            // fp32 pays most for (64 rows of 50,257 x 768: 16 waves 46 us, 4 waves
            // 65; one row of 151,936 x 2,048 bf16: 132 and 123 us); 8 to 16 of
            // them, as many as fill the last round of workgroups best.
            constexpr int kWide = 256 / sizeof(T);  // 256 bytes of a row a step: 116 us, 128 bytes 122, 512 bytes 120
            int waves = a.N <= 4 ? 4 : 8;  // 16 rows of 151,936 x 1,024: 8 waves 62 us, 4 waves 66; one row of 2,048: 117 and 115
            if (a.N > 16) {
                int64_t least = INT64_MAX;
                for (int w = 16; w >= 8; --w) {
                    const int64_t c = (int64_t)tiles_of(tiles_of(a.V, w * 16), kCUs) * w;
                    if (c < least) {
                        least = c;
                        waves = w;
                    }
                }
            }
            const unsigned wgs = (unsigned)tiles_of(a.V, waves * 16), threads = waves * 64;
            if (a.N <= 16) head_stream_kernel<T, 1, 4, 8, kWide><<<dim3(wgs), threads, 0, st>>>(a);
            else if (a.N <= 32) head_stream_kernel<T, 2, 8, 16, 64><<<dim3(wgs), threads, 0, st>>>(a);
            else head_stream_kernel<T, 4, 8, 16, 64><<<dim3(wgs), threads, 0, st>>>(a);
            if (wgs > 1) head_join_kernel<<<dim3((unsigned)a.N), 1024, 0, st>>>(a, a.N, (int)wgs, 1, false);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            continue;
        }
        hipError_t e = pack_rows<T>(a, cap, dtype == GR_BF16 ? kPackPlanes : kPackHalves, false, st);
        if (e != hipSuccess) return e;
        const Shape shape = cut_logits<T>(a.V, a.N, a.D).shape;
        const int step = reads_in_place(a.weight, a.wstride, a.D, dtype) ? a.V : a.plan.Vw;
        for (int v = 0; v < a.V; v += step) {
            const int nv = a.V - v < step ? a.V - v : step;
            const Operand W = words_operands<T>(a, v, nv, false, dtype, st).logits;
            if (shape == kLarge) run_parts<typename LogitTile<T, kLarge>::type>(a, W, cap, v, nv, st);
            else if (shape == kSmall) run_parts<typename LogitTile<T, kSmall>::type>(a, W, cap, v, nv, st);
            else run_parts<typename LogitTile<T, kDeep>::type>(a, W, cap, v, nv, st);
        }
        const int parts = tiles_of(a.V, shape == kLarge ? LogitTile<T, kLarge>::type::WM : LogitTile<T, kSmall>::type::WM);
        int rb = 256;  // four threads to a row, more where it has many parts
        while (rb > 16 && parts > 8 * (1024 / rb)) rb /= 2;
        head_join_kernel<<<dim3((unsigned)tiles_of(a.N, rb)), 1024, 0, st>>>(a, cap, parts, rb, true);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename Tile>
void run_grad(const HeadArgs& a, const Operand& W, int64_t cap, int v, int nv, hipStream_t st) {
    head_grad_kernel<Tile><<<dim3((unsigned)(tiles_of(nv, Tile::BM) * tiles_of(a.N, Tile::BN))), Tile::NT, 0, st>>>(a, W, cap, v, nv);
}

template <typename T, typename Tile>
void run_ghidden(const HeadArgs& a, const Operand& W, int64_t cap, int v, int nv, int splits, hipStream_t st) {
    const int tiles = tiles_of(a.D, Tile::BM) * tiles_of(a.N, Tile::BN);
    head_ghidden_kernel<T, Tile><<<dim3((unsigned)(tiles * splits)), Tile::NT, 0, st>>>(a, W, cap, nv, splits, v == 0,
                                                                                       splits == 1 && v + nv == a.V);
}

template <typename T, typename Tile>
void run_gweight(const HeadArgs& a, int64_t cap, int v, int nv, int splits, hipStream_t st) {
    const int tiles = tiles_of(a.D, Tile::BM) * tiles_of(nv, Tile::BN);
    head_gweight_kernel<T, Tile><<<dim3((unsigned)(tiles * splits)), Tile::NT, 0, st>>>(a, cap, v, nv, splits);
    if (splits > 1) head_gweight_out_kernel<T><<<dim3((unsigned)nv), 256, 0, st>>>(a, v, nv, splits);
}

// One launch: up to kSmallMost rows and words, and no more work for the busiest
// workgroup than the other way's launches cost.  Loss and backward together:
// fp32 256 x 256 x 256 70 us against 102, 500 x 500 x 256 103 against 107 (three
// planes cost the other way more); bf16 48 x 48 x 64 36 against 48, 256 x 256 x
// 256 56 against 50.
bool small_backward(const HeadArgs& a, int dtype) {
    const int64_t most = a.N > a.V ? a.N : a.V;
    return most <= kSmallMost && most * a.D <= (dtype == GR_BF16 ? 32 << 10 : 128 << 10);
}

// Cost of the three products of a piece of `words` words.
template <typename T>
double piece_cost(int64_t rows, int64_t words, int64_t dim) {
    return cut_logits<T>(words, rows, dim).cost + cut_gradient<T, false>(dim, rows, words).cost +
           cut_gradient<T, true>(dim, words, rows).cost;
}

template <typename T>
hipError_t head_backward_t(const HeadArgs& a, int dtype, hipStream_t st) {
    if (small_backward(a, dtype)) {
        const int row_wgs = a.ghidden ? tiles_of(a.N, 16) : 0, word_wgs = a.gweight ? tiles_of(a.V, 16) : 0;
        const int most = a.N > a.V ? a.N : a.V;
        const size_t lds = 16 * (size_t)(tiles_of(most, 16) * 16 + 4) * sizeof(float);
        head_small_backward_kernel<T><<<dim3((unsigned)(row_wgs + word_wgs)), 256, lds, st>>>(a, row_wgs);
        return hipGetLastError();
    }
    const int64_t cap = a.plan.packed;
    const bool in_place = reads_in_place(a.weight, a.wstride, a.D, dtype);
    const int step = in_place || a.plan.Vg < a.plan.Vw ? a.plan.Vg : a.plan.Vw;
    // grad_hidden's cut serves all pieces (their sums meet): the first is the largest
    const Cut hc = cut_gradient<T, false>(a.D, a.N, a.V < step ? a.V : step);
    const hipError_t e = pack_rows<T>(a, cap, dtype == GR_BF16 ? kPackPlanes : kPackHalves + (a.gweight ? kPackPlanes : 0),
                                      a.ghidden && hc.splits == 1, st);
    if (e != hipSuccess) return e;
    for (int v = 0; v < a.V; v += step) {
        const int nv = a.V - v < step ? a.V - v : step;
        const Words W = words_operands<T>(a, v, nv, a.ghidden != nullptr, dtype, st);
        const Shape z = cut_logits<T>(nv, a.N, a.D).shape;
        if (z == kLarge) run_grad<typename LogitTile<T, kLarge>::type>(a, W.logits, cap, v, nv, st);
        else if (z == kSmall) run_grad<typename LogitTile<T, kSmall>::type>(a, W.logits, cap, v, nv, st);
        else run_grad<typename LogitTile<T, kDeep>::type>(a, W.logits, cap, v, nv, st);
        if (a.ghidden) {
            if (hc.shape == kLarge) run_ghidden<T, typename TileFor<T, true, false, kLarge>::type>(a, W.planes, cap, v, nv, hc.splits, st);
            else if (hc.shape == kSmall) run_ghidden<T, typename TileFor<T, true, false, kSmall>::type>(a, W.planes, cap, v, nv, hc.splits, st);
            else run_ghidden<T, typename TileFor<T, true, false, kDeep>::type>(a, W.planes, cap, v, nv, hc.splits, st);
        }
        if (a.gweight) {
            const Cut c = cut_gradient<T, true>(a.D, nv, a.N);
            if (c.shape == kLarge) run_gweight<T, typename TileFor<T, true, true, kLarge>::type>(a, cap, v, nv, c.splits, st);
            else if (c.shape == kSmall) run_gweight<T, typename TileFor<T, true, true, kSmall>::type>(a, cap, v, nv, c.splits, st);
            else run_gweight<T, typename TileFor<T, true, true, kDeep>::type>(a, cap, v, nv, c.splits, st);
        }
    }
    if (a.ghidden && hc.splits > 1) head_ghidden_out_kernel<T><<<dim3((unsigned)a.N), 256, 0, st>>>(a, hc.splits);
    return hipGetLastError();
}

}  // namespace

HeadPlan head_plan(int64_t max_rows, int64_t vocab, int64_t dim, int dtype, bool backward) {
    const auto round_up = [](int64_t x, int64_t to) { return (x + to - 1) / to * to; };
    HeadPlan p{};
    p.planes = dtype == GR_BF16 ? 1 : 3;
    p.Dp = (int32_t)round_up(dim, 8);
    p.part_rows = (int32_t)(max_rows < kPartRows ? max_rows : kPartRows);
    p.packed = backward ? max_rows : p.part_rows;
    const int64_t words = round_up(vocab, kWordTile);
    p.halves = dtype == GR_BF16 ? 0 : 2;
    const int64_t vw = kTableElems / (p.planes + p.halves) / p.Dp / kWordTile * kWordTile;
    p.Vw = (int32_t)(vw < kWordTile ? kWordTile : (vw < words ? vw : words));
    p.W = (int64_t)p.planes * p.Vw * p.Dp;
    p.parts = (vocab + kPartWords - 1) / kPartWords * (int64_t)p.part_rows;
    if (backward) {
        const int64_t vg = kPieceElems / p.planes / max_rows / kWordTile * kWordTile;
        // fp32 and odd rows: the table's piece is packed; a row of G is an operand's
        const int64_t fit = vg < p.Vw ? vg : p.Vw, whole = words < kMaxTileStride ? words : kMaxTileStride;
        const int64_t most_words = fit < kWordTile ? kWordTile : (fit < whole ? fit : whole);
        // the fewest pieces or up to four more, whichever fills the chip best
        const int64_t fewest = (words + most_words - 1) / most_words;
        double least = 1e300;
        for (int64_t pieces = fewest; pieces <= fewest + 4; ++pieces) {
            const int64_t vg = round_up((words + pieces - 1) / pieces, kWordTile), last = words - (words - 1) / vg * vg;
            const auto cost = [&](int64_t w) {
                return dtype == GR_BF16 ? piece_cost<uint16_t>(max_rows, w, dim) : piece_cost<float>(max_rows, w, dim);
            };
            const double c = (double)((words - 1) / vg) * cost(vg) + cost(last);
            if (c < least * 0.999) {
                least = c;
                p.Vg = (int32_t)vg;
            }
        }
        p.G = (int64_t)p.planes * max_rows * p.Vg;
        // a split product has at most kMostRounds rounds of tiles (cut_product)
        const int64_t most = (int64_t)kMostRounds * kCUs * 256 * 256;
        const int64_t h = max_rows * p.Dp, w = (int64_t)p.Vg * p.Dp;
        p.gh = h > most ? h : (h * kMaxSplits < most ? h * kMaxSplits : most);
        p.gw = w * kMaxSplits < most ? w * kMaxSplits : most;
    }
    return p;
}

hipError_t launch_head_loss(const HeadArgs& a, int dtype, hipStream_t st) {
    if (a.N == 0) return hipSuccess;
    return dtype == GR_BF16 ? head_loss_t<uint16_t>(a, dtype, st) : head_loss_t<float>(a, dtype, st);
}

hipError_t launch_head_backward(const HeadArgs& a, int dtype, hipStream_t st) {
    if (a.N == 0) {
        if (a.accumulate || !a.gweight) return hipSuccess;
        if (dtype == GR_BF16) head_zero_kernel<uint16_t><<<dim3((unsigned)a.V), 256, 0, st>>>(a);
        else head_zero_kernel<float><<<dim3((unsigned)a.V), 256, 0, st>>>(a);
        return hipGetLastError();
    }
    return dtype == GR_BF16 ? head_backward_t<uint16_t>(a, dtype, st) : head_backward_t<float>(a, dtype, st);
}

}  // namespace gr
