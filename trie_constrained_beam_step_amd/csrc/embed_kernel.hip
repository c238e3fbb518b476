// embed_kernel.hip -- rows of the embedding table for a step's tokens, and the
// table's gradient from those rows' gradient.
//
// Both move rows and add little: they are bound by HBM.  A row is read and
// written 16 bytes a thread, `lanes` threads to a row.
//
// The gradient has one writer per word and no floating-point atomics.  Few
// tokens (embed_few_kernel): one launch, each workgroup collects its words'
// tokens itself.  More: a stable sort of the token positions by word (its
// launches also fill the gradient with zeros), then every `tile` neighbours in
// the sorted order are summed by one group of threads; a word that lies inside
// one tile is written at once, the sums of one that crosses tiles are joined in
// order by a last kernel.  The order of every sum depends on the tokens alone.
#include "device_common.h"
#include "gr.h"
#include "vocab.h"

namespace gr {
namespace {

typedef float f32x4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint16_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// 16 bytes of a row's elements, kElems of them; `left` of the row's exist.  Raw is
// how they are loaded, value(raw, e) element e as fp32.  Rows need no alignment
// beyond the element's: the hardware takes 16-byte accesses anywhere.
template <typename T>
struct Pack;
template <>
struct Pack<float> {
    static constexpr int kElems = 4;
    typedef f32x4v Raw;
    typedef f32x4v Anywhere __attribute__((aligned(4)));
    static __device__ __forceinline__ Raw raw(const float* p, int left) {
        if (left >= 4) return *(const Anywhere*)p;
        Raw r = {};
        #pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < left) r[e] = p[e];
        return r;
    }
    static __device__ __forceinline__ float value(const Raw& r, int e) { return r[e]; }
    static __device__ __forceinline__ void store(float* p, int left, const float (&x)[4]) {
        if (left >= 4) {
            *(Anywhere*)p = f32x4v{x[0], x[1], x[2], x[3]};
            return;
        }
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < left) p[e] = x[e];
    }
};
template <>
struct Pack<uint16_t> {
    static constexpr int kElems = 8;
    typedef u32x4 Raw;
    typedef u32x4 Anywhere __attribute__((aligned(2)));
    static __device__ __forceinline__ Raw raw(const uint16_t* p, int left) {
        if (left >= 8) return *(const Anywhere*)p;
        Raw r = {};
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < left) r[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
        return r;
    }
    static __device__ __forceinline__ float value(const Raw& r, int e) {
        return __uint_as_float(e & 1 ? r[e >> 1] & 0xFFFF0000u : r[e >> 1] << 16);
    }
    static __device__ __forceinline__ void store(uint16_t* p, int left, const float (&x)[8]) {
        if (left >= 8) {
            u32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = bf16_bits(x[2 * e]) | (uint32_t)bf16_bits(x[2 * e + 1]) << 16;
            *(Anywhere*)p = v;
            return;
        }
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < left) p[e] = bf16_bits(x[e]);
    }
};

// Writes a word's sum: scaled, or added to what its row holds.
template <typename T, int N = Pack<T>::kElems>
__device__ __forceinline__ void put_word(const EmbedBackwardArgs& a, int v, int d, float (&s)[N]) {
    T* o = (T*)a.gweight + (int64_t)v * a.wstride + d;
    if (a.accumulate) {
        const typename Pack<T>::Raw old = Pack<T>::raw(o, a.D - d);
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] = fmaf(s[e], a.scale, Pack<T>::value(old, e));
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] *= a.scale;
    }
    Pack<T>::store(o, a.D - d, s);
}

template <typename T, int N = Pack<T>::kElems>
__device__ __forceinline__ void add_row(const EmbedBackwardArgs& a, int i, int d, float (&s)[N]) {
    const typename Pack<T>::Raw x = Pack<T>::raw((const T*)a.grad + (int64_t)i * a.gstride + d, a.D - d);
#pragma unroll
    for (int e = 0; e < N; ++e) s[e] += Pack<T>::value(x, e);
}

constexpr int kFewWords = 512;  // words of an embed_few_kernel workgroup at most

__device__ __forceinline__ bool in_table(int t, int V) { return (uint32_t)t < (uint32_t)V; }

// --------------------------------------------------------------- lookup

// 256 / lanes groups of `lanes` threads, each R rows at a time: their tokens,
// then their elements, are loaded together.  16,384 rows of 2,048 bf16: 17 us,
// 67 MB written; hot words' rows come from the caches.
template <typename T, int R>
__global__ __launch_bounds__(256) void embed_lookup_kernel(EmbedLookupArgs a, int lanes) {
    constexpr int N = Pack<T>::kElems;
    const int group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    const int64_t i0 = ((int64_t)blockIdx.x * (256 / lanes) + group) * R;
    int t[R];
#pragma unroll
    for (int r = 0; r < R; ++r) t[r] = i0 + r < a.n ? a.tokens[i0 + r] : -1;
    for (int d = (blockIdx.y * lanes + lane) * N; d < a.D; d += gridDim.y * lanes * N) {
        typename Pack<T>::Raw x[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (in_table(t[r], a.V)) x[r] = Pack<T>::raw((const T*)a.weight + (int64_t)t[r] * a.wstride + d, a.D - d);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (i0 + r >= a.n) break;
            float y[N];
#pragma unroll
            for (int e = 0; e < N; ++e) y[e] = in_table(t[r], a.V) ? Pack<T>::value(x[r], e) * a.scale : 0.0f;
            Pack<T>::store((T*)a.out + (i0 + r) * a.ostride + d, a.D - d, y);
        }
    }
}

// ------------------------------------------------------- few tokens, one launch

// 48 tokens of 48 words, 64 wide: 5 us, a chain of loads and LDS passes.
// A workgroup owns the words [x*words, (x+1)*words).  It lists the positions of
// its words' tokens in order, ranks them by word (counting the better ones in
// LDS: the list is short), and its groups of threads take the words in turn.
template <typename T>
__global__ __launch_bounds__(256) void embed_few_kernel(EmbedBackwardArgs a, int lanes, int words) {
    constexpr int N = Pack<T>::kElems;
    __shared__ int pos[kEmbedFew], word[kEmbedFew], sorted[kEmbedFew], wcount[4];
    __shared__ int first[kFewWords], count[kFewWords];
    const int v0 = blockIdx.x * words, nv = min(words, a.V - v0);
    const int wave = threadIdx.x >> 6;
    for (int v = threadIdx.x; v < nv; v += 256) count[v] = 0;
    int m = 0;
    for (int i0 = 0; i0 < a.n; i0 += 256) {
        const int i = i0 + threadIdx.x;
        const int t = i < a.n ? a.tokens[i] : -1;
        const bool mine = t >= v0 && t < v0 + nv;
        const uint64_t b = __ballot(mine);
        if ((threadIdx.x & 63) == 0) wcount[wave] = __popcll(b);
        __syncthreads();
        int at = m + lanes_below(b);
        for (int w = 0; w < wave; ++w) at += wcount[w];
        if (mine) {
            pos[at] = i;
            word[at] = t - v0;
        }
        m += wcount[0] + wcount[1] + wcount[2] + wcount[3];
        __syncthreads();
    }
    for (int q = threadIdx.x; q < m; q += 256) {
        const int v = word[q];
        int below = 0, same = 0;
        for (int r = 0; r < m; ++r) {
            below += word[r] < v ? 1 : 0;
            same += word[r] == v && r < q ? 1 : 0;
        }
        sorted[below + same] = pos[q];
        if (same == 0) first[v] = below;
        atomicAdd(&count[v], 1);
    }
    __syncthreads();
    const int groups = 256 / lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    for (int v = group; v < nv; v += groups) {
        const int c = count[v], f = c ? first[v] : 0;
        if (c == 0 && a.accumulate) continue;
        for (int d = lane * N; d < a.D; d += lanes * N) {
            float s[N] = {};
#pragma unroll 4
            for (int q = 0; q < c; ++q) add_row<T>(a, sorted[f + q], d, s);
            put_word<T>(a, v0 + v, d, s);
        }
    }
}

// ---------------------------------------------------------------- the sort

// A stable radix sort of positions by word, kSortBits at most a pass; tokens
// outside the table sort as word V, behind all others.  A pass: digits counted
// per workgroup of kSortChunk positions; each digit's counts summed over the
// workgroups; positions moved, ranked within a wave by matching lanes and
// between waves by the waves' counts.  163,840 tokens of 1,280 words, one pass:
// 5 + 5 + 11 us, chains of dependent loads; larger chunks (fewer workgroups)
// were slower, 4,096 positions 11 + 5 + 21 us.
constexpr int kSortThreads = 256, kSortWaves = kSortThreads / 64;
constexpr int kSortRounds = kSortChunk / kSortThreads;

__device__ __forceinline__ int word_of(const EmbedBackwardArgs& a, int t) { return in_table(t, a.V) ? t : a.V; }

// The zeros under the gradient's rows are written beside the sort, whose own
// work leaves most of the chip idle: each of its launches carries a share of
// the fill as further workgroups.  On 16,384 tokens of 151,936 words (311 MB of
// zeros) that hides the sort behind the fill.
struct Fill {
    int first;      // fill workgroup of this launch's first
    int64_t rows;   // of a fill workgroup
    int32_t size;   // bytes of an element
};

__device__ void fill_zeros(const EmbedBackwardArgs& a, const Fill& f, int wg) {
    const int64_t r0 = (int64_t)(f.first + wg) * f.rows, r1 = min((int64_t)a.V, r0 + f.rows);
    typedef u32x4 Anywhere __attribute__((aligned(2)));
    const auto zeros = [&](char* o, int64_t bytes) {
        for (int64_t i = (int64_t)threadIdx.x * 16; i + 16 <= bytes; i += blockDim.x * 16) *(Anywhere*)(o + i) = u32x4{0, 0, 0, 0};
        const int64_t end = bytes / 16 * 16 + (int64_t)threadIdx.x * 2;  // elements are of two bytes or four
        if (end < bytes) *(uint16_t*)(o + end) = 0;
    };
    char* o = (char*)a.gweight + r0 * a.wstride * f.size;
    if (a.wstride == a.D) {  // one run
        zeros(o, (r1 - r0) * a.D * f.size);
        return;
    }
    for (int64_t r = r0; r < r1; ++r, o += a.wstride * f.size) zeros(o, (int64_t)a.D * f.size);
}

__global__ __launch_bounds__(kSortThreads) void embed_count_kernel(EmbedBackwardArgs a, const int32_t* keys, int nb, int shift,
                                                                   int digits, Fill fill) {
    extern __shared__ int hist[];  // [digits]
    if ((int)blockIdx.x >= nb) return fill_zeros(a, fill, blockIdx.x - nb);
    for (int d = threadIdx.x; d < digits; d += kSortThreads) hist[d] = 0;
    __syncthreads();
    const int base = blockIdx.x * kSortChunk;
#pragma unroll 4
    for (int r = 0; r < kSortRounds; ++r) {
        const int i = base + r * kSortThreads + threadIdx.x;
        if (i < a.n) atomicAdd(&hist[((keys ? keys[i] : word_of(a, a.tokens[i])) >> shift) & (digits - 1)], 1);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kSortThreads) a.ws.table[(int64_t)blockIdx.x * digits + d] = hist[d];
}

// Each digit's counts over the workgroups become the counts before them: 16
// digits to a workgroup, 16 threads to a digit, each a run of the workgroups.
constexpr int kScanDigits = 16, kScanRuns = 16;

__global__ __launch_bounds__(kScanDigits * kScanRuns) void embed_scan_kernel(EmbedBackwardArgs a, int nb, int digits, int own,
                                                                             Fill fill) {
    __shared__ int sums[kScanRuns][kScanDigits];
    if ((int)blockIdx.x >= own) return fill_zeros(a, fill, blockIdx.x - own);
    const int c = threadIdx.x % kScanDigits, run = threadIdx.x / kScanDigits, d = blockIdx.x * kScanDigits + c;
    const int per = (nb + kScanRuns - 1) / kScanRuns, b0 = run * per, b1 = min(nb, b0 + per);
    int sum = 0;
    if (d < digits)
#pragma unroll 8
        for (int b = b0; b < b1; ++b) sum += a.ws.table[(int64_t)b * digits + d];
    sums[run][c] = sum;
    __syncthreads();
    int before = 0, total = 0;
    for (int r = 0; r < kScanRuns; ++r) {
        before += r < run ? sums[r][c] : 0;
        total += sums[r][c];
    }
    if (d >= digits) return;
    if (run == 0) a.ws.totals[d] = total;
#pragma unroll 8
    for (int b = b0; b < b1; ++b) {
        int32_t* p = a.ws.table + (int64_t)b * digits + d;
        const int x = *p;
        *p = before;
        before += x;
    }
}

__global__ __launch_bounds__(kSortThreads) void embed_move_kernel(EmbedBackwardArgs a, const int32_t* keys, const int32_t* from,
                                                                  int32_t* keys_out, int32_t* to, int nb, int shift,
                                                                  int bits, Fill fill) {
    extern __shared__ int at[];  // [waves][digits]
    __shared__ int wsum[kSortWaves];
    if ((int)blockIdx.x >= nb) return fill_zeros(a, fill, blockIdx.x - nb);
    const int digits = 1 << bits, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (int d = threadIdx.x; d < digits; d += kSortThreads)
        for (int w = 0; w < kSortWaves; ++w) at[(w << bits) + d] = 0;
    __syncthreads();
    // a wave's positions are consecutive: kSortRounds of 64
    const int base = blockIdx.x * kSortChunk + wave * (kSortChunk / kSortWaves);
    int key[kSortRounds];
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const int i = base + r * 64 + lane;
        key[r] = i < a.n ? (keys ? keys[i] : word_of(a, a.tokens[i])) : -1;
        if (i < a.n) atomicAdd(&at[(wave << bits) + ((key[r] >> shift) & (digits - 1))], 1);
    }
    __syncthreads();
    // where each wave's first position of each digit goes
    constexpr int kRounds = (1 << kSortBits) / kSortThreads;
    int totals[kRounds], counts[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int d = r * kSortThreads + threadIdx.x;
        totals[r] = d < digits ? a.ws.totals[d] : 0;
        counts[r] = d < digits ? a.ws.table[(int64_t)blockIdx.x * digits + d] : 0;
    }
    int carry = 0;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int d = r * kSortThreads + threadIdx.x;
        if (r * kSortThreads >= digits) break;
        const int total = totals[r];
        const int inc = (int)wave_inclusive_scan((uint32_t)total);
        if (lane == 63) wsum[wave] = inc;
        __syncthreads();
        int before = carry + inc - total;
        for (int w = 0; w < wave; ++w) before += wsum[w];
        for (int w = 0; w < kSortWaves; ++w) carry += wsum[w];
        if (d < digits) {
            int o = before + counts[r];
            for (int w = 0; w < kSortWaves; ++w) {
                const int c = at[(w << bits) + d];
                at[(w << bits) + d] = o;
                o += c;
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const int i = base + r * 64 + lane;
        const bool ok = i < a.n;
        const int d = (key[r] >> shift) & (digits - 1);
        uint64_t same = __ballot(ok);
        for (int b = 0; b < bits; ++b) {
            const uint64_t one = __ballot((d >> b) & 1);
            same &= (d >> b) & 1 ? one : ~one;
        }
        const int rank = lanes_below(same);
        int o = 0;
        if (ok) o = at[(wave << bits) + d];
        __builtin_amdgcn_wave_barrier();  // every lane has read before the first of a digit moves its place on
        if (ok && rank == 0) at[(wave << bits) + d] = o + __popcll(same);
        __builtin_amdgcn_wave_barrier();
        if (ok) {
            keys_out[o + rank] = key[r];
            to[o + rank] = from ? from[i] : i;
        }
    }
}

// At most kSortFew positions: one workgroup sorts (word, position) pairs in LDS,
// the others are the fill.  One launch for six, against a workgroup alone on its
// network; the whole backward of fp32 rows of 256, 4,212 words: 600 tokens 23.5 us
// against 34.9 by the radix sort, 2,048 32 against 35, 4,096 49 against 37.
constexpr int kSortFewThreads = 1024;

__global__ __launch_bounds__(kSortFewThreads) void embed_sort_few_kernel(EmbedBackwardArgs a, int P, Fill fill) {
    extern __shared__ __align__(16) uint64_t ent[];  // [P], a power of two
    if (blockIdx.x > 0) return fill_zeros(a, fill, blockIdx.x - 1);
    for (int i = threadIdx.x; i < P; i += kSortFewThreads)
        ent[i] = i < a.n ? (uint64_t)(uint32_t)word_of(a, a.tokens[i]) << 32 | (uint32_t)i : ~0ull;
    __syncthreads();
    block_bitonic_sort<kSortFewThreads, false>(ent, P);
    for (int i = threadIdx.x; i < a.n; i += kSortFewThreads) {
        a.ws.keys[0][i] = (int32_t)(ent[i] >> 32);
        a.ws.pos[0][i] = (int32_t)(uint32_t)ent[i];
    }
}

// ---------------------------------------------------------------- the sums

// Bound by reading the rows: 163,840 of 512 fp32 in 58 us, 5.5 TB/s, eight rows in
// flight a thread and the next eight's words and positions with them.
// Group g sums the sorted positions [g*tile, (g+1)*tile), word after word.
// Sums of a word that lies in the tile are written; the tile's part of one that
// began before it goes to part 0 of the tile, of one that goes on behind it to
// part 1 (to part 0 if it did both).
// Whole: a group is whole waves, so its words are the same in every lane of a
// wave and the branches on them are scalar.
template <typename T, bool Whole>
__global__ __launch_bounds__(256) void embed_sum_kernel(EmbedBackwardArgs a, const int32_t* __restrict__ keys,
                                                        const int32_t* __restrict__ pos, int lanes, int tile, int tiles) {
    constexpr int N = Pack<T>::kElems;
    const auto uniform = [](int x) { return Whole ? __builtin_amdgcn_readfirstlane(x) : x; };
    const int g = uniform(blockIdx.x * (256 / lanes) + threadIdx.x / lanes), lane = threadIdx.x % lanes;
    if (g >= tiles) return;
    const int i0 = g * tile, i1 = min(a.n, i0 + tile);
    const int before = uniform(i0 > 0 ? keys[i0 - 1] : -1), behind = uniform(i1 < a.n ? keys[i1] : a.V);
    constexpr int kAhead = 8;
    for (int d = lane * N; d < a.D; d += lanes * N) {
        float s[N] = {};
        const auto end_word = [&](int v, bool at_end) {  // the tile's last position of v is summed
            const bool began = v == before, goes_on = at_end && v == behind;
            if (began || goes_on) {
                float* p = a.ws.parts + ((int64_t)g * 2 + (began ? 0 : 1)) * a.Dp + d;
#pragma unroll
                for (int e = 0; e < N; ++e) p[e] = s[e];
            } else {
                put_word<T>(a, v, d, s);
            }
#pragma unroll
            for (int e = 0; e < N; ++e) s[e] = 0.0f;
        };
        int v = uniform(keys[i0]);
        int kn[kAhead], pn[kAhead];  // the next round's words and positions
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            kn[u] = i0 + u < i1 ? keys[i0 + u] : a.V;
            pn[u] = i0 + u < i1 ? pos[i0 + u] : 0;
        }
        for (int i = i0; i < i1 && v < a.V; i += kAhead) {
            typename Pack<T>::Raw x[kAhead];
            int k[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                k[u] = uniform(kn[u]);
                if (k[u] < a.V) x[u] = Pack<T>::raw((const T*)a.grad + (int64_t)uniform(pn[u]) * a.gstride + d, a.D - d);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int q = i + kAhead + u;
                kn[u] = q < i1 ? keys[q] : a.V;
                pn[u] = q < i1 ? pos[q] : 0;
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (k[u] != v && v < a.V) end_word(v, i + u >= i1);
                v = k[u];
                if (v < a.V) {
#pragma unroll
                    for (int e = 0; e < N; ++e) s[e] += Pack<T>::value(x[u], e);
                }
            }
        }
        if (v < a.V) end_word(v, true);  // the tile ended with a round
    }
}

// The words that cross tiles: workgroup g takes the one that begins in tile g
// and goes on behind it.  Its groups of threads each add a run of the tiles'
// parts in order, and the runs' sums are added in order.
constexpr int kJoinThreads = 512;

template <typename T>
__global__ __launch_bounds__(kJoinThreads) void embed_join_kernel(EmbedBackwardArgs a, const int32_t* keys, int lanes, int tile,
                                                                  int tiles) {
    constexpr int N = Pack<T>::kElems;
    __shared__ float runs[kJoinThreads * N];
    const int g = blockIdx.x;
    const int i0 = g * tile, i1 = i0 + tile;
    if (i1 >= a.n) return;
    const int v = keys[i1 - 1];
    if (v >= a.V || keys[i1] != v || (i0 > 0 && keys[i0 - 1] == v)) return;
    // v reaches tile `last`, not tile `over`: most words end soon
    int last = g + 1, over = g + 2;
    while (over < tiles && keys[over * tile] == v) {
        last = over;
        over = min(tiles, g + 2 * (over - g));
    }
    while (over - last > 1) {
        const int mid = (last + over) / 2;
        if (keys[mid * tile] == v) last = mid;
        else over = mid;
    }
    const int groups = kJoinThreads / lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    const int per = (last - g + groups) / groups;  // of the parts g .. last
    const int q0 = g + group * per, q1 = min(last + 1, q0 + per);
    for (int d0 = 0; d0 < a.D; d0 += lanes * N) {
        const int d = d0 + lane * N;
        float s[N] = {};
        if (d < a.D) {
#pragma unroll 8
            for (int q = q0; q < q1; ++q) {
                const float* x = a.ws.parts + ((int64_t)q * 2 + (q == g ? 1 : 0)) * a.Dp + d;
#pragma unroll
                for (int e = 0; e < N; ++e) s[e] += x[e];
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < N; ++e) runs[e * kJoinThreads + threadIdx.x] = s[e];
        __syncthreads();
        if (group == 0 && d < a.D) {
            for (int r = 1; r < groups; ++r)
#pragma unroll
                for (int e = 0; e < N; ++e) s[e] += runs[e * kJoinThreads + r * lanes + lane];
            put_word<T>(a, v, d, s);
        }
    }
}

// ------------------------------------------------------------------ host

// Threads to a row of `chunks` loads: a power of two, at most 256.
int lanes_for(int chunks) {
    int l = 1;
    while (l < chunks && l < 256) l *= 2;
    return l;
}

template <typename T>
hipError_t lookup_t(const EmbedLookupArgs& a, hipStream_t st) {
    constexpr int N = Pack<T>::kElems;
    const int lanes = lanes_for((a.D + N - 1) / N), groups = 256 / lanes;
    // four rows a group once that still leaves several workgroups to a CU
    const int per = a.n >= 4 * 2048 * groups ? 4 : 1;
    const dim3 grid((unsigned)((a.n + (int64_t)groups * per - 1) / (groups * per)));
    if (per == 4) embed_lookup_kernel<T, 4><<<grid, 256, 0, st>>>(a, lanes);
    else embed_lookup_kernel<T, 1><<<grid, 256, 0, st>>>(a, lanes);
    return hipGetLastError();
}

template <typename T>
hipError_t backward_t(const EmbedBackwardArgs& a, hipStream_t st) {
    constexpr int N = Pack<T>::kElems;
    const int chunks = (a.D + N - 1) / N;
    const int lanes = lanes_for(chunks), groups = 256 / lanes;
    if (a.n <= kEmbedFew) {
        // about 32 KB of the gradient to a workgroup
        int words = (int)((32 << 10) / ((int64_t)a.D * sizeof(T)));
        words = words < groups ? groups : (words < kFewWords ? words : kFewWords);
        embed_few_kernel<T><<<dim3((unsigned)((a.V + words - 1) / words)), 256, 0, st>>>(a, lanes, words);
        return hipGetLastError();
    }
    const EmbedPlan p = embed_plan(a.n, a.V, lanes);
    // fill workgroups of about 128 KB, spread over the sort's launches
    const int64_t row_bytes = (int64_t)a.D * sizeof(T);
    Fill f{0, ((128 << 10) + row_bytes - 1) / row_bytes, (int32_t)sizeof(T)};
    const int fills = a.accumulate ? 0 : (int)((a.V + f.rows - 1) / f.rows);
    int launch = 0;
    const auto share = [&]() {  // sets f.first, returns the launch's fill workgroups
        f.first = (int)((int64_t)fills * launch / (3 * p.passes));
        ++launch;
        return (int)((int64_t)fills * launch / (3 * p.passes)) - f.first;
    };
    const int32_t *keys = nullptr, *pos = nullptr;
    if (a.n <= kSortFew) {
        int P = 1;
        while (P < a.n) P *= 2;
        embed_sort_few_kernel<<<dim3((unsigned)(1 + fills)), kSortFewThreads, P * sizeof(uint64_t), st>>>(a, P, f);
        keys = a.ws.keys[0];
        pos = a.ws.pos[0];
    } else {
        for (int q = 0; q < p.passes; ++q) {
            const int shift = q * p.bits, out = q & 1, digits = 1 << p.bits, scans = (digits + kScanDigits - 1) / kScanDigits;
            int more = share();
            embed_count_kernel<<<dim3((unsigned)(p.blocks + more)), kSortThreads, digits * sizeof(int), st>>>(a, keys, p.blocks, shift, digits, f);
            more = share();
            embed_scan_kernel<<<dim3((unsigned)(scans + more)), kScanDigits * kScanRuns, 0, st>>>(a, p.blocks, digits, scans, f);
            more = share();
            embed_move_kernel<<<dim3((unsigned)(p.blocks + more)), kSortThreads, kSortWaves * digits * sizeof(int), st>>>(
                a, keys, pos, a.ws.keys[out], a.ws.pos[out], p.blocks, shift, p.bits, f);
            keys = a.ws.keys[out];
            pos = a.ws.pos[out];
        }
    }
    const dim3 grid((unsigned)((p.tiles + groups - 1) / groups));
    if (lanes >= 64) embed_sum_kernel<T, true><<<grid, 256, 0, st>>>(a, keys, pos, lanes, p.tile, p.tiles);
    else embed_sum_kernel<T, false><<<grid, 256, 0, st>>>(a, keys, pos, lanes, p.tile, p.tiles);
    embed_join_kernel<T><<<dim3((unsigned)p.tiles), kJoinThreads, 0, st>>>(a, keys, lanes, p.tile, p.tiles);
    return hipGetLastError();
}

}  // namespace

EmbedPlan embed_plan(int64_t n, int64_t vocab, int lanes) {
    EmbedPlan p{};
    int bits = 1;
    while ((vocab >> bits) > 0) ++bits;  // words 0 .. vocab
    p.passes = (bits + kSortBits - 1) / kSortBits;
    p.bits = (bits + p.passes - 1) / p.passes;
    p.blocks = (int)((n + kSortChunk - 1) / kSortChunk);
    // small tiles spread the rows over the chip (2^18 threads fill it), large
    // ones leave fewer parts to join and bound their memory
    p.tile = 8;
    while (n * lanes / (2 * p.tile) >= (1 << 18) || (n + p.tile - 1) / p.tile > kSumTiles) p.tile *= 2;
    p.tiles = (int)((n + p.tile - 1) / p.tile);
    return p;
}

hipError_t launch_embed_lookup(const EmbedLookupArgs& a, int dtype, hipStream_t st) {
    if (a.n == 0) return hipSuccess;
    return dtype == GR_BF16 ? lookup_t<uint16_t>(a, st) : lookup_t<float>(a, st);
}

hipError_t launch_embed_backward(const EmbedBackwardArgs& a, int dtype, hipStream_t st) {
    if (a.n == 0 && a.accumulate) return hipSuccess;
    return dtype == GR_BF16 ? backward_t<uint16_t>(a, st) : backward_t<float>(a, st);
}

}  // namespace gr
