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
// Planes.  An fp32 operand is held as three bf16 planes, x = x0 + x1 + x2, each
// the bf16 nearest to what the ones before it leave: 8 significant bits a
// plane, so the sum is x itself.  A product takes the six pairs of planes whose
// index sum is at most two; the three left out are below 2^-23 |a b|.  Six
// bf16 products run 2.8 times as fast as one fp32 product on these cores
// (dense peaks 2.5 PFLOP/s against 157 TFLOP/s, over six).
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

// BM x BN tile, waves of WM x WN, BK deep (32 or 64), PL planes.
template <int BM_, int BN_, int WM_, int WN_, int BK_, int PL_, bool AAcross, bool BAcross>
struct GemmTile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = BK_, PL = PL_;
    static constexpr int NT = (BM / WM) * (BN / WN) * 64;
    static constexpr int FM = WM / 16, FN = WN / 16;
    static constexpr bool kPerm = !AAcross;  // rows of A are interleaved (frag_row)
    static constexpr int ABytes = BM * BK * 2, BBytes = BN * BK * 2;  // a plane's
    static constexpr int Stage = PL * (ABytes + BBytes);

    // Copies one operand's R x BK tile (all planes) into LDS.  `base` is the
    // tile's first element, `rem` the bytes from there to the operand's end,
    // kleft the k elements left.
    template <int R, bool Across, bool Perm>
    static __device__ __forceinline__ void fetch(char* lds, const uint16_t* base, int64_t ld, int64_t plane, int64_t rem,
                                                 int kleft) {
        constexpr int kRowChunks = Across ? R / 8 : BK / 8;
        constexpr int kRowsPerRound = NT / kRowChunks;
        constexpr int kRounds = R * BK * 2 / (NT * 16);
        static_assert(R * BK * 2 % (NT * 16) == 0, "whole rounds");
        static_assert(kRowsPerRound % 16 == 0, "the swizzle repeats from round to round");
        const int tid = threadIdx.x;
        const int row = tid / kRowChunks, c = tid % kRowChunks;
        uint32_t off;
        if (Across) {
            off = (uint32_t)row * (uint32_t)(ld * 2) + (uint32_t)(c ^ (across_swz(row) << 1)) * 16u;
        } else {
            const int src = c ^ along_swz<kRowChunks, Perm>(row);
            off = (uint32_t)row * (uint32_t)(ld * 2) + (uint32_t)src * 16u;
            if (src * 8 >= kleft) off = 0x80000000u;  // behind the last k: zero
        }
        const uint32_t step = (uint32_t)kRowsPerRound * (uint32_t)(ld * 2);
        const uint32_t n = rem > 0x7FFFFFFF ? 0x7FFFFFFFu : (rem > 0 ? (uint32_t)rem : 0u);
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
#pragma unroll
        for (int pl = 0; pl < PL; ++pl) {
            const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)(base + pl * plane), 0, n, kBufferFlags);
#pragma unroll
            for (int r = 0; r < kRounds; ++r)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rsrc, (lds_void*)(lds + pl * R * BK * 2 + r * NT * 16 + wave * 1024), 16, off + r * step, 0, 0, 0);
        }
    }

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

    static __device__ __forceinline__ void multiply(const char* lds, f32x4v (&acc)[FM][FN]) {
        const int wave = threadIdx.x >> 6;
        const int rm = (wave / (BN / WN)) * WM, rn = (wave % (BN / WN)) * WN;
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk) {
            bf16x8 a[PL][FM], b[PL][FN];
#pragma unroll
            for (int pl = 0; pl < PL; ++pl) {
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    const char* s = lds + PL * ABytes + pl * BBytes;
                    b[pl][j] = BAcross ? frag_across<BN>(s, rn, j, kk) : frag_along<false>(s, rn, j, kk);
                }
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const char* s = lds + pl * ABytes;
                    a[pl][i] = AAcross ? frag_across<BM>(s, rm, i, kk) : frag_along<kPerm>(s, rm, i, kk);
                }
            }
            // the small pairs first
#pragma unroll
            for (int sum = PL - 1; sum >= 0; --sum)
#pragma unroll
                for (int pa = sum; pa >= 0; --pa)
#pragma unroll
                    for (int i = 0; i < FM; ++i)
#pragma unroll
                        for (int j = 0; j < FN; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[pa][i], b[sum - pa][j], acc[i][j], 0, 0, 0);
        }
    }

    // Waits for this wave's loads into LDS and its reads of it, then for the
    // workgroup's.
    static __device__ __forceinline__ void stage_barrier() {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }

    // acc += the tile at rows m0 of A and n0 of B, k in [k0, k1).  s0, s1: two
    // stages of LDS.  k0 is a multiple of 8 and k1 of BK, or what lies behind
    // k1 is zero in one operand and finite in the other (rows behind an
    // "across" operand's end are zero).
    static __device__ __forceinline__ void run(const Operand& A, int64_t m0, const Operand& B, int64_t n0, int64_t k0,
                                               int64_t k1, char* s0, char* s1, f32x4v (&acc)[FM][FN]) {
        const auto load = [&](char* lds, int64_t k) {
            const int kleft = (int)(k1 - k < BK ? k1 - k : BK);
            const int64_t ao = AAcross ? k * A.ld + m0 : m0 * A.ld + k;
            const int64_t bo = BAcross ? k * B.ld + n0 : n0 * B.ld + k;
            fetch<BM, AAcross, kPerm>(lds, A.p + ao, A.ld, A.plane, (A.n - ao) * 2, kleft);
            fetch<BN, BAcross, false>(lds + PL * ABytes, B.p + bo, B.ld, B.plane, (B.n - bo) * 2, kleft);
        };
        if (k0 >= k1) return;
        load(s0, k0);
        stage_barrier();
        for (int64_t k = k0; k < k1; k += 2 * BK) {
            if (k + BK < k1) load(s1, k + BK);
            multiply(s0, acc);
            stage_barrier();
            if (k + BK >= k1) break;
            if (k + 2 * BK < k1) load(s0, k + 2 * BK);
            multiply(s1, acc);
            stage_barrier();
        }
    }
};

}  // namespace
}  // namespace gr
