// gemm_tile.h -- one workgroup's tile of C[m][n] = sum_k A[m][k] B[n][k] on the
// matrix cores, from bf16 operands in global memory into fp32 accumulators.
//
// Operands.  An operand lies in memory either with its k index contiguous
// ("along": element (r, k) at p[r*ld + k]) or with its row index contiguous
// ("across": (r, k) at p[k*ld + r]).  Both are copied to LDS as they lie, 16
// bytes a lane, by the buffer loads that write LDS directly; an "across" tile
// is turned on the way to registers by the transposing LDS read
// (ds_read_b64_tr_b16: 16 lanes read four k rows of 16 elements, and lane i
// gets the four of column i).  So one table serves W, W^T, H, H^T, G and G^T.
//
// Planes.  An fp32 operand is held in planes of 16 bits, x = x0 + x1 (+ x2), each
// the nearest to what the ones before it leave; a product takes the pairs of
// planes whose index sum is below their number, and sums them in fp32.  fp32
// matrix instructions run at 157 TFLOP/s, 16-bit ones at 2.5 PFLOP/s.
//   three bf16 planes, six pairs: 8 significant bits a plane, so the sum is x
//     itself, over the whole range of fp32; the pairs left out are below 2^-23
//     |a b|.
//   two fp16 planes, three pairs (Half): 11 bits a plane leave x0 + x1 within
//     2^-22 of x, if x is between 2^-14 and 2^16: for operands whose rows can
//     be scaled by a power of two that divides out of the product again (the
//     logits' both; 2^15 is put on a row's largest element, and elements down
//     to 2^-17 of it keep their 22 bits, smaller ones are off by 2^-40 of the
//     largest).  With the pair left out a product is off by 3 * 2^-22 |a b| at
//     most, a few roundings of an fp32 sum.
//
// Bounds.  Every load goes through a buffer descriptor that ends with the
// operand, so rows behind its last one read as zero.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gr {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4v __attribute__((ext_vector_type(4)));

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

struct Operand {
    const uint16_t* p;  // 16-byte aligned
    int64_t ld;         // elements, a multiple of 8, at most kMaxTileStride
    int64_t plane;      // elements between planes
    int64_t n;          // elements from p to the operand's end, a multiple of 8
};

// 256 rows of this stride stay below 2^30 bytes: offsets inside a tile are 32 bits
constexpr int64_t kMaxTileStride = 1 << 20;

constexpr uint32_t kBufferFlags = 0x00020000;  // raw buffer, 32-bit data

// The 16-byte chunk of an "along" row (Chunks of them) is stored at its index
// xor this, so that the 16 rows of a fragment read start in different banks.
// Perm: the rows of a fragment are 8*q + r, r < 4 (see frag_row).
template <int Chunks, bool Perm>
__device__ __forceinline__ int along_swz(int row) {
    if (Chunks == 8) return Perm ? ((row & 3) | ((row >> 1) & 4)) : (row & 7);
    return Perm ? (((row >> 1) & 1) | ((row >> 2) & 2)) : ((row >> 1) & 3);
}
// The same for the 32-byte pieces of an "across" row k.
__device__ __forceinline__ int across_swz(int k) { return (k & 3) | ((k >> 1) & 4); }

// Rows of A's fragment `t`, lane row i (0..15).  Perm: two neighbouring
// fragments interleave so that a lane's four accumulators of each are eight
// consecutive rows: row = 32*(t/2) + 8*(i/4) + 4*(t%2) + i%4.
template <bool Perm>
__device__ __forceinline__ int frag_row(int t, int i) {
    return Perm ? (t >> 1) * 32 + (i >> 2) * 8 + (t & 1) * 4 + (i & 3) : t * 16 + i;
}

// One step of the matrix cores on 16 x 16 x 32 elements of either 16-bit type.
template <bool Half>
__device__ __forceinline__ f32x4v mfma16(bf16x8 a, bf16x8 b, f32x4v c) {
    typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
    if (Half) return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// BM x BN tile, waves of WM x WN, BK deep (32 or 64), PL planes (Half: of fp16),
// ST stages of LDS.
template <int BM_, int BN_, int WM_, int WN_, int BK_, int PL_, bool AAcross, bool BAcross, bool Half_ = false, int ST_ = 2>
struct GemmTile {
    static constexpr bool Half = Half_;
    static constexpr int ST = ST_;
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = BK_, PL = PL_;
    static constexpr int NT = (BM / WM) * (BN / WN) * 64;
    static constexpr int FM = WM / 16, FN = WN / 16;
    // the waves take turns (see turns()): eight waves, two to a SIMD, whose "across"
    // fragments take twice the LDS reads of "along" ones.  Measured at 2,048 x
    // 16,384 x 7,424 (grad_weight's) 1,235 TFLOP/s against 1,094 in step, at
    // 32,768 x 7,424 x 2,048 (the logits', both "along") 1,160 against 1,253.
    static constexpr bool kTurns = AAcross && NT == 512;
    static_assert(!kTurns || ST == 2, "turns take two stages");
    static constexpr bool kPerm = !AAcross;  // rows of A are interleaved (frag_row)
    static constexpr int ABytes = BM * BK * 2, BBytes = BN * BK * 2;  // a plane's
    static constexpr int Stage = PL * (ABytes + BBytes);
    static constexpr int Lds = ST * Stage;

    // Copies one operand's R x BK tile (all planes) into LDS, one k step after
    // the other.
    template <int R, bool Across, bool Perm>
    struct Fetch {
        static constexpr int kRowChunks = Across ? R / 8 : BK / 8;
        static constexpr int kRowsPerRound = NT / kRowChunks;
        static constexpr int kRounds = R * BK * 2 / (NT * 16);
        static_assert(R * BK * 2 % (NT * 16) == 0, "whole rounds");
        static_assert(kRowsPerRound % 16 == 0, "the swizzle repeats from round to round");
        const char* base;  // the next step's first element
        int64_t rem;       // bytes from there to the operand's end
        int64_t plane, advance;
        uint32_t off, step;
        int kfirst;        // "along": this lane's first k in a step

        __device__ __forceinline__ Fetch(const Operand& o, int64_t r0, int64_t k0) {
            const int row = threadIdx.x / kRowChunks, c = threadIdx.x % kRowChunks;
            const int src = Across ? c ^ (across_swz(row) << 1) : c ^ along_swz<kRowChunks, Perm>(row);
            const int64_t first = Across ? k0 * o.ld + r0 : r0 * o.ld + k0;
            base = (const char*)(o.p + first);
            rem = (o.n - first) * 2;
            plane = o.plane * 2;
            advance = (Across ? o.ld : 1) * BK * 2;
            off = (uint32_t)row * (uint32_t)(o.ld * 2) + (uint32_t)src * 16u;
            step = (uint32_t)kRowsPerRound * (uint32_t)(o.ld * 2);
            kfirst = Across ? 0 : src * 8;
        }

        // kleft: the k elements left from this step on.  `wave_lds`: the stage's
        // place for this operand, plus the wave's 1 KB.
        __device__ __forceinline__ void operator()(char* wave_lds, int kleft) {
            const uint32_t n = rem > 0x7FFFFFFF ? 0x7FFFFFFFu : (rem > 0 ? (uint32_t)rem : 0u);
            uint32_t o = Across || kfirst < kleft ? off : 0x80000000u;  // behind the last k: zero
#pragma unroll
            for (int r = 0; r < kRounds; ++r, o += step)
#pragma unroll
                for (int pl = 0; pl < PL; ++pl)
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(
                        __builtin_amdgcn_make_buffer_rsrc((void*)(base + pl * plane), 0, n, kBufferFlags),
                        (lds_void*)(wave_lds + pl * R * BK * 2 + r * NT * 16), 16, o, 0, 0, 0);
            base += advance;
            rem -= advance;
        }
    };

    // Fragment (16 rows x 32 k) of an "along" tile.
    template <bool Perm>
    static __device__ __forceinline__ bf16x8 frag_along(const char* lds, int r0, int t, int kk) {
        const int lane = threadIdx.x & 63;
        const int row = r0 + frag_row<Perm>(t, lane & 15);
        const int c = (kk * 4 + (lane >> 4)) ^ along_swz<BK / 8, Perm>(row);
        return *(const bf16x8*)(lds + row * BK * 2 + c * 16);
    }

    // The same of an "across" tile of R rows.
    template <int R>
    static __device__ __forceinline__ bf16x8 frag_across(const char* lds, int r0, int t, int kk) {
        const int lane = threadIdx.x & 63;
        const int k = kk * 32 + (lane >> 4) * 8 + ((lane & 15) >> 2);
        const int piece = ((r0 >> 4) + t) ^ across_swz(k);
        const char* a = lds + k * R * 2 + piece * 32 + (lane & 3) * 8;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)a);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a + 4 * R * 2));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }

    // The fragments of step s (k half s / FM, A's fragment s % FM) are read two
    // steps before their matrix instructions, and the half's B fragments with
    // its first: the order is fixed, or the compiler reads a whole stage ahead
    // and spills.
    static __device__ __forceinline__ void multiply(const char* lds, f32x4v (&acc)[FM][FN]) {
        const int wave = threadIdx.x >> 6;
        const int rm = (wave / (BN / WN)) * WM, rn = (wave % (BN / WN)) * WN;
        constexpr int kSteps = BK / 32 * FM, kAhead = 2;
        bf16x8 a[kAhead + 1][PL], b[2][PL][FN];
        const auto read = [&](int s) {
            const int kk = s / FM, i = s % FM;
#pragma unroll
            for (int pl = 0; pl < PL; ++pl) {
                if (i == 0)
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        const char* t = lds + PL * ABytes + pl * BBytes;
                        b[kk & 1][pl][j] = BAcross ? frag_across<BN>(t, rn, j, kk) : frag_along<false>(t, rn, j, kk);
                    }
                const char* t = lds + pl * ABytes;
                a[s % (kAhead + 1)][pl] = AAcross ? frag_across<BM>(t, rm, i, kk) : frag_along<kPerm>(t, rm, i, kk);
            }
        };
#pragma unroll
        for (int s = 0; s < kAhead; ++s) read(s);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            if (s + kAhead < kSteps) read(s + kAhead);
            __builtin_amdgcn_sched_barrier(0);
            // the small pairs of planes first
#pragma unroll
            for (int sum = PL - 1; sum >= 0; --sum)
#pragma unroll
                for (int pa = sum; pa >= 0; --pa)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        acc[s % FM][j] = mfma16<Half>(a[s % (kAhead + 1)][pa], b[(s / FM) & 1][sum - pa][j], acc[s % FM][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // Waits for this wave's reads of LDS, and for its loads into LDS too if
    // `loads`, then for the workgroup's.
    static __device__ __forceinline__ void stage_barrier(bool loads) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        if (loads) __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
        else __builtin_amdgcn_s_waitcnt(0xC07F);        // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }

    // acc += the tile at rows m0 of A and n0 of B, k in [k0, k1).  lds: the
    // stages.  k0 is a multiple of 8 and k1 of BK, or what lies behind k1 is
    // zero in one operand and finite in the other (rows behind an "across"
    // operand's end are zero).
    static __device__ __forceinline__ void run(const Operand& A, int64_t m0, const Operand& B, int64_t n0, int k0, int k1,
                                               char* lds, f32x4v (&acc)[FM][FN]) {
        if (k0 >= k1) return;
        Fetch<BM, AAcross, kPerm> fa(A, m0, k0);
        Fetch<BN, BAcross, false> fb(B, n0, k0);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        char* wave_lds = lds + wave * 1024;
        const int steps = (k1 - k0 + BK - 1) / BK;
        const auto load = [&](int i) {
            char* to = wave_lds + i % ST * Stage;
            fa(to, k1 - k0 - i * BK);
            fb(to + PL * ABytes, k1 - k0 - i * BK);
        };
        if (kTurns) {
            load(0);
            turns(lds, steps, wave >= NT / 128, load, acc);
        } else {
            together(lds, steps, load, acc);
        }
    }

    // All waves in step: ST - 1 steps are in flight before the first, and each
    // issues the loads of the one ST - 1 behind it at its start, into the stage
    // that the step before it has read.  Its own loads are the oldest but those
    // of ST - 2 steps.
    template <typename Load>
    static __device__ __forceinline__ void together(const char* lds, int steps, const Load& load, f32x4v (&acc)[FM][FN]) {
        constexpr int kYounger = (ST - 2) * PL * (ABytes + BBytes) / (NT * 16);  // loads of a wave
        static_assert(kYounger < 64, "the wait counts up to 63");
        for (int i = 0; i < ST - 1; ++i)
            if (i < steps) load(i);
        for (int i = 0; i < steps; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("" ::: "memory");
            // vmcnt(kYounger), or (0) where fewer steps are in flight; lgkmcnt(0)
            if (i + ST - 2 < steps) __builtin_amdgcn_s_waitcnt((kYounger & 15) | (kYounger >> 4) << 14 | 0x0070);
            else __builtin_amdgcn_s_waitcnt(0x0070);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            if (i + ST - 1 < steps) load(i + ST - 1);
            __builtin_amdgcn_s_setprio(1);
            multiply(lds + i % ST * Stage, acc);
            __builtin_amdgcn_s_setprio(0);
        }
    }

    // The two waves of a SIMD take turns: while one reads its fragments of a
    // whole step, the other's matrix instructions run.  Half of the waves
    // (`second`) are a phase behind; phase 2i is the first half's reads of step
    // i and the second half's products of step i - 1, phase 2i + 1 the other way
    // round.  Step i + 1 is loaded by all in phase 2i (its stage was last read
    // in phase 2i - 1) and waited for at the end of phase 2i + 1.
    template <typename Load>
    static __device__ __forceinline__ void turns(const char* lds, int steps, bool second, const Load& load,
                                                 f32x4v (&acc)[FM][FN]) {
        const int wave = threadIdx.x >> 6;
        const int rm = (wave / (BN / WN)) * WM, rn = (wave % (BN / WN)) * WN;
        constexpr int kHalves = BK / 32;
        stage_barrier(true);
        if (second) {
            if (steps > 1) load(1);
            stage_barrier(false);
        }
        for (int i = 0; i < steps; ++i) {
            const char* st = lds + (i & 1) * Stage;
            if (!second && i + 1 < steps) load(i + 1);
            bf16x8 a[kHalves][PL][FM], b[kHalves][PL][FN];
#pragma unroll
            for (int kk = 0; kk < kHalves; ++kk)
#pragma unroll
                for (int pl = 0; pl < PL; ++pl) {
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        const char* t = st + PL * ABytes + pl * BBytes;
                        b[kk][pl][j] = BAcross ? frag_across<BN>(t, rn, j, kk) : frag_along<false>(t, rn, j, kk);
                    }
#pragma unroll
                    for (int q = 0; q < FM; ++q) {
                        const char* t = st + pl * ABytes;
                        a[kk][pl][q] = AAcross ? frag_across<BM>(t, rm, q, kk) : frag_along<kPerm>(t, rm, q, kk);
                    }
                }
            stage_barrier(second);
            if (second && i + 2 < steps) load(i + 2);
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int kk = 0; kk < kHalves; ++kk)
#pragma unroll
                for (int sum = PL - 1; sum >= 0; --sum)
#pragma unroll
                    for (int pa = sum; pa >= 0; --pa)
#pragma unroll
                        for (int q = 0; q < FM; ++q)
#pragma unroll
                            for (int j = 0; j < FN; ++j)
                                acc[q][j] = mfma16<Half>(a[kk][pa][q], b[kk][sum - pa][j], acc[q][j]);
            __builtin_amdgcn_s_setprio(0);
            stage_barrier(!second);
        }
        if (!second) stage_barrier(false);
    }
};

}  // namespace
}  // namespace gr
