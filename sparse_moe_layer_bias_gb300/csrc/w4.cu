// w4.cu -- products of a few tokens with 4-bit weights and group scales: one
// matrix (lmoe_w4_matvec), and the routed experts of a decode batch
// (lmoe_w4_experts; the 4-bit path of lmoe_forward).
//
//   w[r][c] = (u[r][c] - 8) * s[r][c / g],  u in 0..15 (two to a byte, the even
//   column in the low half), s bf16, g = 32, 64 or 128
//   y[t][r] = sum over c of x[t][c] w[r][c] = sum over groups of s * (sum of (u - 8) x)
//
// The weights are read once, in the caller's row-major layout, and everything
// else is small: the kernels are bound by HBM, and next by the ALU that takes the
// codes apart.  The inner sums run on mma.sync m16n8k16 (16 weight rows x 8
// columns): u - 8 is exact in fp16, x is taken to fp16 by a power of two that
// brings the largest of a token's values in the warp's columns (in
// w4_rows_kernel, of its row) to 2^14..2^15 (which cuts off at most 2^-35 of it: half of
// the columns are held divided by 16, the others lose 2^-39), the products are exact and are
// summed in fp32, and each group's sum is scaled in fp32 afterwards, so nothing
// is rounded below fp32.  (fp16 rather than bf16 because its 10 bits of mantissa
// take two codes out of one shifted word: 5 ALU operations for 8 codes instead of
// 7.  tcgen05.mma would need the weights as 16-bit values in shared memory, four
// times the bytes written back through it; a warp's own mma takes them from
// registers.)  The experts' activations are fp32 and enter W3 the same way, rounded to
// fp16's 11 bits: 2^-12 of each, a sixteenth of what z's rounding to bf16 may take.
// Two fp16 halves would keep them whole, for twice the mma.
//
// Two kernels share this: w4_kernel, whose warps split a row's columns, and further down
// w4_rows_kernel, whose warps take whole rows; which one a call takes is said at
// w4_wants_maps and w4_entry_rows.
//
// w4_kernel.  A warp's task is 16 rows x 512 columns (4 blocks of 128): 4 KB of codes that
// cp.async brings into one of the warp's two slots, two tasks ahead.  A block's
// codes lie there as 16-byte chunks (one row, 32 columns), so that ldmatrix
// hands lane (r, q) the 8 codes of row r, columns 8q.. of a group of 32: the A
// fragment of two mma, up to the order of the columns within the 8, in which
// the x fragments are put to match (0 4 1 5 2 6 3 7).
//
// A warp keeps to its columns: its x fragments are loaded once and stay while row
// tile after row tile streams past, so a weight's way is HBM -> shared memory ->
// registers -> mma and x costs nothing per tile.  With P < 8 tokens at a time the
// mma's 8 columns hold the tokens 8 / P times over, each time with another part of
// the 512 columns: the x fragments take 8 P registers instead of 64, and of a
// group's products only the columns that hold its part are added up.  The warps of
// a block that share a row tile add their sums through shared memory.  For one token
// the time is latency, not bandwidth: a token's 16 of 896 experts (3584 x 512, group 32) take
// 27.8 us in two launches, 49.6 MB; 14336 x 1024 by one row 6.0 us, 8.3 MB.
// (Tasks half as wide, for twice the warps: no faster, 28.5 us against 28.5 then.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace lmoe {

namespace {

constexpr int kMaxWarps = 16;
constexpr int kTaskCols = 512;
constexpr int kScaleStride = 40;   // bytes between the rows of a slot's scales
constexpr int kSlotBytes = 4096 + 16 * kScaleStride;
constexpr int kSlots = 2;

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// d = a b + c (no side effects, so the compiler may order them freely)
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// Eight codes -> fp16 pairs (u0, u4) - 8, 16 ((u1, u5) - 8), (u2, u6) - 8, 16 ((u3, u7) - 8).
// 0x6400 | v is 1024 + v in fp16 for v < 1024, so the subtractions are exact; the
// x that meet the odd pairs are divided by 16.
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t (&p)[4]) {
    const __half2 off = __floats2half2_rn(1032.f, 1032.f), off16 = __floats2half2_rn(1152.f, 1152.f);
    const uint32_t w8 = w >> 8;
    uint32_t v[4];
    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(v[0]) : "r"(w));
    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(v[1]) : "r"(w));
    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(v[2]) : "r"(w8));
    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(v[3]) : "r"(w8));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 d = __hsub2(*reinterpret_cast<__half2 *>(&v[i]), i & 1 ? off16 : off);
        p[i] = *reinterpret_cast<const uint32_t *>(&d);
    }
}

// A row's sum, or NaN where it is infinite through one of the row's scales: the weights of such a
// group are NaN.  (An infinite scale meets a group's sum that is 0 in one form and a rounding's residue
// in another, so that the row's sum is NaN or an infinity, of which the softcaps would make a finite
// number.)  The scales are looked at again for infinite sums only, so it costs nothing while the
// weights stream past: within 1% in every case.
__device__ __forceinline__ float settle(float v, const uint16_t *scales, int ng) {
    if (fabsf(v) == __int_as_float(0x7f800000)) {
#pragma unroll 1
        for (int g = 0; g < ng; ++g)
            if ((scales[g] & 0x7fffu) == 0x7f80u) v = __int_as_float(0x7fffffff);
    }
    return v;
}

// A matrix of 4-bit weights: n rows of k columns.
struct Mat {
    const uint8_t *codes;
    const uint16_t *scales;
};
struct MatShape {
    int n, k;
    int64_t ldc;      // bytes between rows of codes (a multiple of 16)
    int64_t lds;      // scales between rows
    int row_bytes;    // bytes of a row that hold codes, up to 16
    int ng;           // groups of a row
    int kt;           // tasks of a row: ceil(k / 512)
    int full;         // of them whole, with scales that copies of 8 bytes may take
    int unit;         // bytes on which every row of scales starts, up to 16
};

// Bring task kt of rows row0.. into a slot (one commit group).
template <int GPB>
__device__ __forceinline__ void fetch_task(uint32_t slot, const Mat &m, const MatShape &sh, int row0, int kt) {
    const int lane = threadIdx.x & 31;
    const int r0 = lane >> 2, chunk = lane & 3;
    constexpr int kRow = 8 * GPB;   // bytes of a row's scales
    const int g0 = kt * 4 * GPB;
    const uint32_t dst = slot + (chunk * 16 + (r0 ^ (2 * chunk))) * 16;   // (row r0 + 8: 128 bytes on)
    const uint32_t sdst = slot + 4096;
    const uint8_t *src = m.codes + int64_t(row0 + r0) * sh.ldc + (kt * 256 + chunk * 16);
    if (row0 + 16 <= sh.n && kt < sh.full) {   // a whole task, and its scales in copies of 8 bytes
#pragma unroll
        for (int b = 0; b < 4; ++b) cp16(dst + b * 1024, src + b * 64, 16);
        src += 8 * sh.ldc;
#pragma unroll
        for (int b = 0; b < 4; ++b) cp16(dst + b * 1024 + 128, src + b * 64, 16);
        constexpr int per = kRow / 8;   // copies of a row: 4, 2, 1
        const int r = lane / per, byte = lane % per * 8;
        const uint8_t *ss = reinterpret_cast<const uint8_t *>(m.scales + int64_t(row0 + r) * sh.lds + g0) + byte;
        const uint32_t sd = sdst + r * kScaleStride + byte;
        if (per > 1 || lane < 16) cp8(sd, ss, 8);
        if (per == 4) cp8(sd + 8 * kScaleStride, ss + 16 * sh.lds, 8);
        cp_commit();
        return;
    }
    const int nr = min(16, sh.n - row0);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const bool ok = r0 + 8 * h < nr && kt * 256 + b * 64 + chunk * 16 < sh.row_bytes;
            cp16(dst + b * 1024 + h * 128, ok ? src + h * 8 * sh.ldc + b * 64 : m.codes, ok ? 16 : 0);
        }
    }
    // 16 rows x 4 * GPB scales, zero where there is none
    auto left = [&](int r, int byte) {   // bytes that exist from here on
        return r < nr ? max(0, (sh.ng - g0) * 2 - byte) : 0;
    };
    if (sh.unit >= 4) {
        const int lg = sh.unit >= 8 ? 3 : 2;
        const int per = kRow >> lg;
        for (int i = lane; i < 16 * per; i += 32) {
            const int r = i / per, byte = (i % per) << lg;
            const int n = min(1 << lg, left(r, byte));
            const uint8_t *ss = n > 0 ? reinterpret_cast<const uint8_t *>(m.scales + int64_t(row0 + r) * sh.lds + g0) + byte
                                      : reinterpret_cast<const uint8_t *>(m.scales);
            if (lg == 3)
                cp8(sdst + r * kScaleStride + byte, ss, n);
            else
                cp4(sdst + r * kScaleStride + byte, ss, n);
        }
    } else {
        constexpr int per = kRow / 2;
        for (int i = lane; i < 16 * per; i += 32) {
            const int r = i / per, g = i % per;
            const uint16_t v = left(r, 2 * g) > 0 ? m.scales[int64_t(row0 + r) * sh.lds + g0 + g] : uint16_t(0);
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(sdst + r * kScaleStride + 2 * g), "h"(v) : "memory");
        }
    }
    cp_commit();
}

// acc = the task's products with the x fragments xf.  Part g / (2 P) of the 16
// groups of 32 columns is in the mma columns from P g / (2 P) on.
template <int P, int GPB>
__device__ __forceinline__ void run_task(uint32_t slot, const uint4 (&xf)[2 * P], float (&acc)[4]) {
    const int lane = threadIdx.x & 31;
    const int n = lane >> 2;
    const int mat = lane >> 3;
    // the lane's chunk of a block's two ldmatrix: (row, chunk of 32 columns)
    const int row = (mat & 1) * 8 + (lane & 7);
    const uint32_t at0 = slot + ((mat >> 1) * 16 + (row ^ (2 * (mat >> 1)))) * 16;
    const uint32_t at1 = slot + ((2 + (mat >> 1)) * 16 + (row ^ (2 * (2 + (mat >> 1))))) * 16;
    const uint32_t sp = slot + 4096 + n * kScaleStride;
    acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        uint32_t w[8], sc[2][2];
        {
            uint32_t t[4];
            ldmatrix4(t, at0 + b * 1024);
            w[0] = t[0], w[1] = t[1], w[2] = t[2], w[3] = t[3];
            ldmatrix4(t, at1 + b * 1024);
            w[4] = t[0], w[5] = t[1], w[6] = t[2], w[7] = t[3];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {   // the block's scales of rows n and n + 8
            const uint32_t p = sp + 8 * h * kScaleStride + b * 2 * GPB;
            if (GPB == 4) {
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(sc[h][0]), "=r"(sc[h][1]) : "r"(p));
            } else if (GPB == 2) {
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(sc[h][0]) : "r"(p));
            } else {
                uint16_t v;
                asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(p));
                sc[h][0] = v;
            }
        }
        float d[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {   // groups of 32 columns; 4 / GPB of them share a scale
            uint32_t lo[4], hi[4];
            unpack8(w[2 * g], lo);
            unpack8(w[2 * g + 1], hi);
            const uint4 x = xf[(b * 4 + g) % (2 * P)];
            if (g % (4 / GPB) == 0)
                mma_f16(d, lo[0], hi[0], lo[1], hi[1], x.x, x.y, 0.f, 0.f, 0.f, 0.f);
            else
                mma_f16(d, lo[0], hi[0], lo[1], hi[1], x.x, x.y, d[0], d[1], d[2], d[3]);
            mma_f16(d, lo[2], hi[2], lo[3], hi[3], x.z, x.w, d[0], d[1], d[2], d[3]);
            if (g % (4 / GPB) == 4 / GPB - 1) {
                const int si = g / (4 / GPB);
                const uint32_t u0 = sc[0][si >> 1], u1 = sc[1][si >> 1];
                const float s0 = __uint_as_float(si & 1 ? u0 & 0xffff0000u : u0 << 16);
                const float s1 = __uint_as_float(si & 1 ? u1 & 0xffff0000u : u1 << 16);
                // this lane's mma columns: 2 (lane % 4) and the next
                if (P == 8 || (lane & 3) * 2 / P == (b * 4 + g) / (2 * P)) {
                    acc[0] = fmaf(s0, d[0], acc[0]);
                    acc[1] = fmaf(s0, d[1], acc[1]);
                    acc[2] = fmaf(s1, d[2], acc[2]);
                    acc[3] = fmaf(s1, d[3], acc[3]);
                }
            }
        }
    }
}

// Eight consecutive columns as fp16 pairs in fragment order, times up (the odd pairs times up / 16).
// An infinity becomes NaN (h * 0 + h), so that its row gives NaN whether the codes are met as u - 8 or
// with their offset, whose surplus comes off as infinity - infinity.
__device__ __forceinline__ uint4 to_fragment(const float (&f)[8], float up) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float u = i & 1 ? up * 0.0625f : up;
        const __half2 v = __floats2half2_rn(f[i] * u, f[i + 4] * u);
        const __half2 h = __hfma2(v, __floats2half2_rn(0.f, 0.f), v);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 to_fragment(uint4 v, float up) {   // of bf16
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return to_fragment(f, up);
}
// 2^(14 - exponent) for the largest magnitude (its fp32 bits), at most 2^126; and its inverse
__device__ __forceinline__ float scale_up(uint32_t top, float &down) {
    const int shift = min(14 + 127 - static_cast<int>(top >> 23), 126);
    down = __int_as_float((127 - shift) << 23);
    return __int_as_float((127 + shift) << 23);
}
// 8 activations, and the larger of m and their finite magnitudes (as bits)
__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
    const float4 u = *reinterpret_cast<const float4 *>(p), v = *reinterpret_cast<const float4 *>(p + 4);
    f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w, f[4] = v.x, f[5] = v.y, f[6] = v.z, f[7] = v.w;
}
__device__ __forceinline__ uint32_t max_finite(uint32_t m, const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = __float_as_uint(f[i]) & 0x7fffffffu;
        if (b < 0x7f800000u) m = max(m, b);
    }
    return m;
}
// The larger of m and the magnitudes (as fp32 bits) of the finite ones of 8 bf16.
__device__ __forceinline__ uint32_t max_finite(uint32_t m, uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = (w[i] << 16) & 0x7fffffffu, hi = w[i] & 0x7fff0000u;
        if (lo < 0x7f800000u) m = max(m, lo);
        if (hi < 0x7f800000u) m = max(m, hi);
    }
    return m;
}
// The same two at a time: with one added to the exponent, infinities and NaN are negative
// as 16-bit integers.  Half the instructions, for the kernel that has many rows to look
// through; in w4_kernel, whose registers are full, it spills (m = 8: 14.8 us against 12.9).
__device__ __forceinline__ uint32_t max_finite_packed(uint4 v) {
    auto up = [](uint32_t w) { return (w & 0x7fff7fffu) + 0x00800080u; };
    const uint32_t t = __vimax3_s16x2(__vimax3_s16x2(0x00800080u, up(v.x), up(v.y)), up(v.z), up(v.w)) - 0x00800080u;
    return max(t << 16, t & 0xffff0000u);
}

// 8 bf16 of a row of k columns from column c on (zeros past the end)
__device__ __forceinline__ uint4 load8(const uint16_t *row, int c, int k, bool vec) {
    if (vec && c + 8 <= k) return __ldg(reinterpret_cast<const uint4 *>(row + c));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (c + 9 <= k) {   // words of two; a row that starts between two words takes five of them
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + c);
        const uint32_t *p = reinterpret_cast<const uint32_t *>(at & ~uintptr_t(3));
        uint32_t v[5];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __ldg(p + e);
        if (at & 2) {
            v[4] = __ldg(p + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = __byte_perm(v[e], v[e + 1], 0x5432);
            return make_uint4(w[0], w[1], w[2], w[3]);
        }
        return make_uint4(v[0], v[1], v[2], v[3]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (c + e < k) w[e >> 1] |= uint32_t(row[c + e]) << (16 * (e & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// SiTU(p1; b1) * softcap(p2; b2)
__device__ __forceinline__ float situ_glu_exact(float p1, float p2, float b1, float b2) {
    return b1 * tanhf(p1 / b1) / (1.f + expf(-p1)) * (b2 * tanhf(p2 / b2));
}

// What a launch computes: a matrix's products; the experts' activations; the
// experts' outputs by assignment; the sum over each token's experts.
enum Mode { MODE_MATVEC = 0, MODE_W12 = 1, MODE_W3_GROUPED = 2, MODE_W3_TOKEN = 3 };

struct W4Args {
    MatShape sh;
    Mat m[2];               // the matrix, or the experts' (W1 and W2)
    int64_t mat_codes, mat_scales;   // bytes / scales from one expert's matrix to the next
    int tiles;              // row tiles of a matrix
    int rt;                 // row tiles of a unit (of each of W1 and W2)
    int cols;               // column tasks of a row tile: sh.kt (W3 by token: of each of the token's experts)
    int cw, rw;             // warps side by side along the columns, and along the rows
    int units;
    // x: rows of bf16 (matvec, W12), or the activations (W3)
    const uint16_t *x;      // (w4_rows_kernel's experts: as w4_prepare_kernel made them, fp16)
    int64_t ldx;
    int m_rows;
    int xvec;
    const float *x_starts, *x_down;
    // routing
    const int32_t *idx;     // [T * k] chosen experts
    int topk, E;
    const int4 *list;       // grouped: {expert, first place in perm, rows, 0}
    const int32_t *n_list;
    const int32_t *perm;    // grouped: assignment at each place
    const float *gates;
    float *act;             // [T * k][act_ld] the experts' activations
    int act_ld;
    float beta1, beta2;
    // results
    void *y;
    int64_t ldy;
    int y_f32;
    float *o;               // W3 grouped: [T * k][n] fp32
    unsigned *err;          // status word of the caller's handle, or nullptr: the library's
};

// A unit is rt row tiles of one matrix (W12: of W1 and of W2; W3 by token: of each of the
// token's experts) for up to P rows of x (the experts': one), so that a block mostly stays
// with the fragments it has.  Warp (c, r) takes column tasks c, c + cw, ... and of each the
// tiles r, r + rw, ...; what it gets for a tile goes to its own place in shared memory, and
// the block sums a tile's cw places in order.
template <int MODE, int P, int GPB, int THREADS>
__global__ void __launch_bounds__(THREADS) __maxnreg__(P == 8 ? 128 : 96) w4_kernel(W4Args a) {
    grid_dependency_wait();
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kPlace = 16 * P;   // floats of a place: [2 halves of the tile x 2 columns][8 rows][P / 2]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cw = a.cw, c_id = warp % cw, r_id = warp / cw;
    const int n_warps = cw * a.rw;
    const uint32_t slots_at = smem_u32(smem) + warp * (kSlots * kSlotBytes);
    float *red0 = reinterpret_cast<float *>(smem + n_warps * kSlots * kSlotBytes);
    const int tiles_u = MODE == MODE_W12 ? 2 * a.rt : a.rt;
    const int red_size = tiles_u * cw * kPlace;
    const int groups = (a.tiles + a.rt - 1) / a.rt;   // units of one matrix
    const int units = a.units;

    // a place in the sequence of this warp's tasks
    struct Cursor {
        int u;
        int entry, expert, tile0;   // of the unit; entry: the token, or the assignment, or matvec's 8 rows
        int col, ti;
    };
    auto open = [&](Cursor &c) {   // the first unit from c.u on that has an expert
        for (; c.u < units; c.u += gridDim.x) {
            c.entry = c.u / groups;
            c.tile0 = (c.u - c.entry * groups) * a.rt;
            c.expert = 0;
            if (MODE == MODE_W12) {
                c.expert = a.idx[c.entry];
                if (c.expert < 0 || c.expert >= a.E) continue;
            }
            break;
        }
    };
    auto rewind = [&](Cursor &c) {   // first task of a unit
        c.col = c_id;
        c.ti = r_id;
    };
    // the next task (every warp has one at least in each unit: c_id < cols, r_id < tiles_u)
    auto advance = [&](Cursor &c) {
        c.ti += a.rw;
        if (c.ti < tiles_u) return;
        c.ti = r_id;
        c.col += cw;
        if (c.col < a.cols) return;
        c.col = c_id;
        c.u += gridDim.x;
        open(c);
    };
    // a task's row tile, its place along the row and its expert (-1: there is no such task)
    auto task = [&](const Cursor &c, int &tile, int &kt) {
        tile = c.tile0 + (MODE == MODE_W12 ? c.ti >> 1 : c.ti);
        kt = c.col;
        int e = c.expert;
        if (MODE == MODE_W3_TOKEN) {
            const int j = c.col / a.sh.kt;
            kt = c.col - j * a.sh.kt;
            e = a.idx[c.entry * a.topk + j];
            if (e < 0 || e >= a.E) e = -1;
        }
        return tile * 16 < a.sh.n ? e : -1;
    };
    auto fetch = [&](Cursor &c, int s) {
        if (c.u < units) {
            int tile, kt;
            const int e = task(c, tile, kt);
            if (e >= 0) {
                Mat m = a.m[MODE == MODE_W12 ? c.ti & 1 : 0];
                if (MODE != MODE_MATVEC) {
                    m.codes += e * a.mat_codes;
                    m.scales += e * a.mat_scales;
                }
                fetch_task<GPB>(slots_at + s * kSlotBytes, m, a.sh, tile * 16, kt);
            } else {
                cp_commit();
            }
            advance(c);
        } else {
            cp_commit();
        }
    };

    Cursor nx;   // the next task to fetch
    nx.u = blockIdx.x;
    open(nx);
    rewind(nx);
    Cursor c = nx;
    fetch(nx, 0);
    fetch(nx, 1);
    int s = 0, buf = 0;
    uint4 xf[2 * P];
    float down0 = 1.f, down1 = 1.f;   // takes the sums of the lane's two columns back
    int x_unit = -1;   // what xf holds
    int x_col = -1;
    while (c.u < units) {
        const int64_t entry = c.entry;
        const int cnt = MODE == MODE_MATVEC ? min(P, a.m_rows - c.entry * P) : 1;
        float *red = red0 + buf * red_size;
        const int u = c.u;
        const int tile0 = c.tile0;
        const int expert = c.expert;
        do {
            int tile, kt;
            const bool there = task(c, tile, kt) >= 0;
            if (c.entry != x_unit || c.col != x_col) {
                x_unit = c.entry;
                x_col = c.col;
                const int n = lane >> 2;   // the fragment's column: token n % P, part n / P
                const int t = n % P;
                const int c8 = kt * kTaskCols + (n / P) * (64 * P) + (lane & 3) * 8;
                uint32_t top = 0;
                float down, up;
                if (MODE == MODE_MATVEC || MODE == MODE_W12) {
                    const uint16_t *row = nullptr;
                    if (t < cnt) row = a.x + (MODE == MODE_MATVEC ? entry * P + t : entry / a.topk) * a.ldx;
#pragma unroll
                    for (int i = 0; i < 2 * P; ++i) {
                        xf[i] = make_uint4(0u, 0u, 0u, 0u);
                        if (row) xf[i] = load8(row, c8 + i * 32, a.sh.k, a.xvec != 0);
                        top = max_finite(top, xf[i]);
                    }
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    up = scale_up(top, down);
#pragma unroll
                    for (int i = 0; i < 2 * P; ++i) xf[i] = to_fragment(xf[i], up);
                } else {
                    const float *row = nullptr;
                    if (there && t == 0) {
                        row = a.act + (entry * a.topk + c.col / a.sh.kt) * a.act_ld;
                    }
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 2 * P; ++i)
                        if (row && c8 + i * 32 < a.act_ld) {
                            load8(row + c8 + i * 32, f);
                            top = max_finite(top, f);
                        }
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    up = scale_up(top, down);
#pragma unroll
                    for (int i = 0; i < 2 * P; ++i) {
                        xf[i] = make_uint4(0u, 0u, 0u, 0u);
                        if (row && c8 + i * 32 < a.act_ld) {
                            load8(row + c8 + i * 32, f);
                            xf[i] = to_fragment(f, up);
                        }
                    }
                }
                down0 = __shfl_sync(0xffffffffu, down, (lane & 3) * 8);
                down1 = __shfl_sync(0xffffffffu, down, (lane & 3) * 8 + 4);
            }
            cp_wait<kSlots - 1>();
            __syncwarp();
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            if (there) run_task<P, GPB>(slots_at + s * kSlotBytes, xf, acc);
            acc[0] *= down0;
            acc[1] *= down1;
            acc[2] *= down0;
            acc[3] *= down1;
            if (MODE == MODE_W3_TOKEN && there) {
                const float g = a.gates[entry * a.topk + c.col / a.sh.kt];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] *= g;
            }
            // the parts' sums together, to the lanes of the first
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (P <= 4) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 2);
                if (P <= 2) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 1);
            }
            if ((lane & 3) < P / 2) {
                float *p = red + (c.ti * cw + c_id) * kPlace + (lane >> 2) * (P / 2) + (lane & 3);
                const bool add = c.col >= cw;
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i * (4 * P)] = add ? p[i * (4 * P)] + acc[i] : acc[i];
            }
            __syncwarp();
            fetch(nx, s);
            s ^= 1;
            advance(c);
        } while (c.u == u);
        __syncthreads();
        buf ^= 1;
        // sum of the places of (tile, row, mma column)
        auto sum = [&](int tile, int row, int col) {
            const float *p = red + tile * cw * kPlace + ((row >> 3) * 2 + (col & 1)) * (4 * P) + (row & 7) * (P / 2) + (col >> 1);
            float v = 0.f;
            for (int i = 0; i < cw; ++i) v += p[i * kPlace];
            return v;
        };
        const int n_out = a.rt * 16;
        for (int i = threadIdx.x; i < n_out * cnt; i += n_warps * 32) {
            const int r = i % n_out, t = i / n_out;
            const int tile = r >> 4, row = tile0 * 16 + r;
            if (MODE == MODE_MATVEC) {
                if (row >= a.sh.n) continue;
                const float v = settle(sum(tile, r & 15, t), a.m[0].scales + int64_t(row) * a.sh.lds, a.sh.ng);
                const int64_t at = (entry * P + t) * a.ldy + row;
                if (a.y_f32)
                    static_cast<float *>(a.y)[at] = v;
                else
                    static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(v);
            } else if (MODE == MODE_W12) {
                if (row >= a.act_ld) continue;
                float act = 0.f;   // features past the last one are zeros
                if (row < a.sh.n) {
                    const int64_t sc = expert * a.mat_scales + int64_t(row) * a.sh.lds;
                    const float p1 = settle(sum(2 * tile, r & 15, t), a.m[0].scales + sc, a.sh.ng);
                    const float p2 = settle(sum(2 * tile + 1, r & 15, t), a.m[1].scales + sc, a.sh.ng);
                    act = situ_glu_exact(p1, p2, a.beta1, a.beta2);
                }
                a.act[entry * a.act_ld + row] = act;
            } else {
                if (row >= a.sh.n) continue;
                float z = sum(tile, r & 15, 0);
                if (fabsf(z) == __int_as_float(0x7f800000)) {
#pragma unroll 1
                    for (int j = 0; j < a.topk; ++j) {
                        const int e = a.idx[entry * a.topk + j];
                        if (e >= 0 && e < a.E) z = settle(z, a.m[0].scales + e * a.mat_scales + int64_t(row) * a.sh.lds, a.sh.ng);
                    }
                }
                if (a.y_f32)
                    static_cast<float *>(a.y)[entry * a.ldy + row] = z;
                else
                    static_cast<__nv_bfloat16 *>(a.y)[entry * a.ldy + row] = __float2bfloat16_rn(z);
            }
        }
    }
    cp_wait<0>();
}

// The same products with whole row tiles to a warp: for many row tiles (a tall matrix, more
// than 8 rows of x, or a batch's experts).  The x rows (up to 8) are in shared memory as fp16 in
// fragment order; a warp walks items of 16 rows x 512 columns, which TMA brings into its two slots
// (two boxes of 128 bytes' width, 128-byte swizzle, so ldmatrix reads without conflicts;
// past the matrix's end it fills zeros) with the item's scales beside them by cp.async.
//
// The row tiles that a block has are one run of items, cut into even ranges, so that its
// warps end together; a tile that is cut has its parts added through shared memory, in order.
// (Whole tiles to a warp: 65536 x 7168 by 8 rows 59 us instead of 53.)  What an SM has on its way
// is 16 warps x 2 slots x 4.6 KB, and while it streams it keeps up with HBM (7 TB/s from the first
// item of a block to its last); what is lost is the start of each unit (its rows of x: 2 to 7 us of
// dependent reads and of conversion), the warps' unequal ends and rounds of units that do not fill
// the blocks.  (Asking for a unit's first items ahead of that by prefetches into L2 made it slower, by
// 1 to 6%: the copies wait behind them.)  Measured: 65536 x 7168 by 8 rows 48 us, 5.1 TB/s;
// 64 tokens of top-16 over 896 experts (3584 x 512) 306 us in five launches, 4.5 TB/s (in some runs
// 328); 6 such tokens 82 us.
//
// Where the result is rounded to bf16 anyway (FAST), the codes are not taken down to
// u - 8: the products with 1024 + u and 16 (64 + u), as they come out of the masks, are
// summed from a start of -(1032 or 72) times the sum of the x that meet them, which is
// computed once with the x rows.  That saves half of the unpacking (a subtraction for
// each pair of codes) and costs bits: the partial sums are up to 225 times the result's
// usual size, so a step of 2^-24 of them is about 2^-16 of it, 2^-7 of a bf16 step.  fp32
// results keep the exact u - 8.
constexpr int kBoxBytes = 2048;           // 16 rows x 256 columns
constexpr int kItemBoxes = 2;
constexpr int kItemCols = 256 * kItemBoxes;
// bytes between rows of an item's scales (rows that start anywhere bring 16 bytes more), and of all
constexpr int scale_row(bool aligned) { return kItemBoxes * 16 + (aligned ? 0 : 16); }
constexpr int item_scales(bool aligned) { return 16 * scale_row(aligned); }
constexpr int kRowsPerSm = 2;             // blocks of 8 warps
constexpr uint64_t kWaitLimitNs = 2000000000ull;        // 2 s per wait for a copy
__device__ unsigned g_w4_status;                        // kDevErrTimeout when a wait of a call without a handle gave up

// (u0, u4), (u1, u5), (u2, u6), (u3, u7) as 1024 + u or, the odd pairs, 16 (64 + u)
__device__ __forceinline__ void unpack8_raw(uint32_t w, uint32_t (&v)[4]) {
    const uint32_t w8 = w >> 8;
    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(v[0]) : "r"(w));
    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(v[1]) : "r"(w));
    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(v[2]) : "r"(w8));
    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(v[3]) : "r"(w8));
}

__device__ __forceinline__ uint32_t lds16(uint32_t at) {
    uint16_t v;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(at));
    return v;
}

// acc += the item's products with the x rows.  row: the lane's ldmatrix row in the first
// box; sp0, sp1: the item's scales of its two rows; xp: its x row at the item's first column;
// cp: the starts of its two columns, twice (as the mma takes them); left: groups of the
// row from the item's first on.
// (With few tokens the mma's spare columns could hold other groups, so that one scaling
// serves several: built for 2 and 4 tokens, it saved a tenth of the instructions and no
// time, the chains of mma being that much longer.)
template <int GPB, bool FAST, bool ALIGNED>
__device__ __forceinline__ void run_item(uint32_t row, uint32_t sp0, uint32_t sp1, uint32_t xp, uint32_t cp, int left,
                                         float (&acc)[4]) {
    constexpr int kOf = 4 / GPB;   // groups of 32 columns that share a scale
    const int r = threadIdx.x & 7, m = (threadIdx.x & 31) >> 4;
    uint32_t off[4];               // of the lane's chunk in a box's four ldmatrix
#pragma unroll
    for (int p = 0; p < 4; ++p) off[p] = ((2 * p + m) ^ r) << 4;
#pragma unroll
    for (int b = 0; b < 2 * kItemBoxes; ++b) {   // blocks of 128 columns
        uint32_t w[8];
        {
            uint32_t t[4];
            ldmatrix4(t, row + (b >> 1) * kBoxBytes + off[2 * (b & 1)]);
            w[0] = t[0], w[1] = t[1], w[2] = t[2], w[3] = t[3];
            ldmatrix4(t, row + (b >> 1) * kBoxBytes + off[2 * (b & 1) + 1]);
            w[4] = t[0], w[5] = t[1], w[6] = t[2], w[7] = t[3];
        }
        float s0[GPB], s1[GPB];   // scales of rows lane / 4 and lane / 4 + 8
        if (GPB == 4 && ALIGNED) {
            uint32_t t[4];
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(t[0]), "=r"(t[1]) : "r"(sp0 + b * 8));
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(t[2]), "=r"(t[3]) : "r"(sp1 + b * 8));
#pragma unroll
            for (int i = 0; i < GPB; ++i) {
                s0[i] = __uint_as_float(i & 1 ? t[i >> 1] & 0xffff0000u : t[i >> 1] << 16);
                s1[i] = __uint_as_float(i & 1 ? t[2 + (i >> 1)] & 0xffff0000u : t[2 + (i >> 1)] << 16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < GPB; ++i) {
                s0[i] = __uint_as_float(lds16(sp0 + (b * GPB + i) * 2) << 16);
                s1[i] = __uint_as_float(lds16(sp1 + (b * GPB + i) * 2) << 16);
            }
        }
        // where the row ends in this item, what lies behind its scales may be anything
#pragma unroll
        for (int i = 0; i < GPB && !ALIGNED; ++i) {
            const bool in = b * GPB + i < left;
            s0[i] = in ? s0[i] : 0.f;
            s1[i] = in ? s1[i] : 0.f;
        }
        float d[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            uint32_t lo[4], hi[4];
            if (FAST) {
                unpack8_raw(w[2 * g], lo);
                unpack8_raw(w[2 * g + 1], hi);
            } else {
                unpack8(w[2 * g], lo);
                unpack8(w[2 * g + 1], hi);
            }
            uint4 x;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                         : "r"(xp + (4 * b + g) * 64));
            if (g % kOf == 0) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                if (FAST)
                    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                                 : "r"(cp + (b * GPB + g / kOf) * 64));
                mma_f16(d, lo[0], hi[0], lo[1], hi[1], x.x, x.y, c[0], c[1], c[2], c[3]);
            } else {
                mma_f16(d, lo[0], hi[0], lo[1], hi[1], x.x, x.y, d[0], d[1], d[2], d[3]);
            }
            mma_f16(d, lo[2], hi[2], lo[3], hi[3], x.z, x.w, d[0], d[1], d[2], d[3]);
            if (g % kOf == kOf - 1) {
                acc[0] = fmaf(s0[g / kOf], d[0], acc[0]);
                acc[1] = fmaf(s0[g / kOf], d[1], acc[1]);
                acc[2] = fmaf(s1[g / kOf], d[2], acc[2]);
                acc[3] = fmaf(s1[g / kOf], d[3], acc[3]);
            }
        }
    }
}

struct RowsArgs {
    W4Args a;       // (m[].codes, mat_codes, rt, cols, cw, rw unused)
    int kt;         // items of a row: ceil(k / 512)
    int xrows;      // x rows in shared memory
    int xstride;    // bytes between them
};

// The sum of the products that the codes' offsets make of a lane's 8 columns (in fragment order).
__device__ __forceinline__ float offset_sum(uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        s[i & 1] += f.x + f.y;
    }
    return fmaf(1032.f, s[0], 1152.f * s[1]);
}

// x rows for w4_rows_kernel (one block each), made once for all the units that read them:
// fp16 in fragment order with zeros up to a whole item, the factor that takes the sums
// back, and the starts of each group of 32 columns.  Of tokens (bf16, ldx apart), and then
// one more block groups the assignments by expert; or of activations (fp32, act_ld apart;
// those of ids outside [0, E) were never written and are left out).
struct PrepArgs {
    const uint16_t *x;
    const float *act;
    int64_t ldx;
    int rows, k, vec, kt;
    uint16_t *xh;
    float *starts, *down;
    const int32_t *idx;
    int n, E, most;
    int32_t *perm;
    int4 *list;
    int32_t *n_list;
};
constexpr int kPrepThreads = 1024;
__device__ __forceinline__ void group_assignments(const int32_t *idx, int n, int E, int most, int32_t *perm,
                                                  int4 *list, int32_t *n_list);
template <bool ACT, int THREADS>
__global__ void __launch_bounds__(THREADS) w4_prepare_kernel(PrepArgs a) {
    grid_dependency_wait();
    const int t = blockIdx.x, lane = threadIdx.x & 31;
    if constexpr (!ACT) {
        if (t == a.rows) {
            group_assignments(a.idx, a.n, a.E, a.most, a.perm, a.list, a.n_list);
            return;
        }
    } else {
        const int e = a.idx[t];
        if (e < 0 || e >= a.E) return;
    }
    __shared__ uint32_t s_top;
    const int chunks = a.kt * (kItemCols / 8);   // (a multiple of a warp)
    auto load = [&](int c, float (&f)[8]) {
        if (ACT) {
            if (c * 8 < a.k)
                load8(a.act + t * a.ldx + c * 8, f);
            else
                f[0] = f[1] = f[2] = f[3] = f[4] = f[5] = f[6] = f[7] = 0.f;
        } else {
            const uint4 v = load8(a.x + t * a.ldx, c * 8, a.k, a.vec != 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    };
    if (threadIdx.x == 0) s_top = 0u;
    __syncthreads();
    uint32_t top = 0;
    float f[8];
    for (int c = threadIdx.x; c < chunks; c += THREADS) {
        load(c, f);
        top = max_finite(top, f);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0 && top) atomicMax(&s_top, top);
    __syncthreads();
    float down;
    const float up = scale_up(s_top, down);
    if (threadIdx.x == 0) a.down[t] = down;
    for (int c = threadIdx.x; c < chunks; c += THREADS) {
        if (c >= THREADS || chunks > THREADS) load(c, f);   // (else they are still there)
        const uint4 h = to_fragment(f, up);
        reinterpret_cast<uint4 *>(a.xh)[int64_t(t) * chunks + c] = h;
        float o = offset_sum(h);
        o += __shfl_xor_sync(0xffffffffu, o, 1);
        o += __shfl_xor_sync(0xffffffffu, o, 2);
        if (lane % 4 == 0) a.starts[int64_t(t) * (chunks / 4) + c / 4] = -o;
    }
}

// Groups that the row tiles are cut into, so that the units' rounds over the blocks take the
// fewest items of a warp, where starting a unit takes as long as kUnitItems.  (A warp's
// lanes try a number each; every warp finds the same.)  Against units of 8 tiles: 3 tokens of
// top-16 over 896 experts 62 -> 55 us, 6 tokens 92 -> 84, 64 tokens 313 -> 308, 64 tokens of top-4 over
// 8 experts 64 -> 48; 16 tokens 155 -> 163.  (kUnitItems 1 or 4: the same within 1%, 16 tokens 164 and 170.)
constexpr int kUnitItems = 2;
__device__ __forceinline__ int tile_groups(int entries, int tiles, int kt, int mats, int warps, int blocks) {
    const int lane = threadIdx.x & 31;
    // 1 to 16, then 16 to 224 in steps of a quarter of a power of two
    const int n = min(tiles, lane < 16 ? lane + 1 : (4 + (lane & 3)) << (lane / 4 - 2));
    const int rounds = (entries * n + blocks - 1) / blocks, unit = (tiles + n - 1) / n;
    const unsigned cost = rounds * ((unit * kt + warps - 1) / warps * mats + kUnitItems);
    const unsigned best = __reduce_min_sync(0xffffffffu, cost * 32 + lane);
    return __shfl_sync(0xffffffffu, n, best & 31);
}

template <int MODE, int GPB, bool FAST, bool ALIGNED, int THREADS>
__global__ void __launch_bounds__(THREADS, 256 * kRowsPerSm / THREADS)
    w4_rows_kernel(const __grid_constant__ W4Maps maps, const __grid_constant__ RowsArgs ra) {
    extern __shared__ __align__(1024) uint8_t smem_rows[];
    uint8_t *smem = smem_rows;
    const W4Args &a = ra.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = blockDim.x >> 5, threads = blockDim.x;
    constexpr int kMats = MODE == MODE_W12 ? 2 : 1;
    constexpr int kScaleRow = scale_row(ALIGNED), kScales = item_scales(ALIGNED);
    // shared memory: code slots, scale slots, x rows, starts, the rows' factors and
    // largest values, their assignments and gates, barriers, the abort flag
    const uint32_t base = smem_u32(smem);
    const uint32_t codes = base + warp * (2 * kItemBoxes * kBoxBytes);
    uint32_t at = warps * (2 * kItemBoxes * kBoxBytes);
    const uint32_t scales = base + at + warp * (2 * kScales);
    at += warps * (2 * kScales);
    uint8_t *xs = smem + at;
    at += ra.xrows * ra.xstride;
    float *starts = reinterpret_cast<float *>(smem + at);   // [groups][4 pairs of columns, each twice]
    at += FAST ? ra.kt * (kItemBoxes * 2 * GPB * 64) : 0;
    float *down = reinterpret_cast<float *>(smem + at);
    uint32_t *top_of = reinterpret_cast<uint32_t *>(smem + at + 32);
    int *as_of = reinterpret_cast<int *>(smem + at + 64), *row_of = as_of + 8;
    float *gate_of = reinterpret_cast<float *>(smem + at + 128);
    float4 *heads = reinterpret_cast<float4 *>(smem + at + 160 + warps * 16 + 16);   // [warp][matrix]: sums of a tile that another warp began
    const uint32_t bars = base + at + 160 + warp * 16;
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + at + 160 + warps * 16);
    auto err = [&] { return a.err ? a.err : &g_w4_status; };
    if (lane < 2) mbar_init(bars + lane * 8, 1);
    if (threadIdx.x == 0) *abort_flag = 0u;
    fence_mbar_init();
    __syncthreads();
    grid_dependency_wait();

    // a unit is an entry (matvec: 8 rows of x) and one of the groups that the row tiles are cut into
    const int tiles = (a.sh.n + 15) / 16;
    const int entries = MODE == MODE_MATVEC ? (a.m_rows + ra.xrows - 1) / ra.xrows : *a.n_list;
    const int groups = MODE == MODE_MATVEC ? gridDim.x / entries : tile_groups(entries, tiles, ra.kt, kMats, warps, gridDim.x);
    const int units = entries * groups;
    // even parts in 32 bits (a division in 64 takes longer than an item): of n, the first n % parts have one more
    const int g_each = tiles / groups, g_more = tiles - g_each * groups;
    auto first_tile = [&](int g) { return g * g_each + min(g, g_more); };
    const int x_chunks = ra.kt * (kItemCols / 8);   // 8-column chunks of an x row
    uint32_t get = 0, use = 0;   // items asked for and used so far: slot n & 1, phase (n >> 1) & 1
    bool dead = false;           // a wait gave up: nothing more is fetched or computed
    int4 ahead = MODE != MODE_MATVEC && int(blockIdx.x) < units ? a.list[blockIdx.x / groups] : int4{};
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        int expert = 0, p0, cnt, g;
        if (MODE == MODE_MATVEC) {   // (all rows of x with the same tiles at about the same time)
            g = u / entries;
            p0 = (u - g * entries) * ra.xrows;
            cnt = min(ra.xrows, a.m_rows - p0);
        } else {
            g = u % groups;
            expert = ahead.x;
            p0 = ahead.y;
            cnt = ahead.z;
            if (u + static_cast<int>(gridDim.x) < units) ahead = a.list[(u + gridDim.x) / groups];   // for the next unit
        }
        // The unit's tiles are one run of steps along their rows (W12: an item of each matrix),
        // cut into even ranges, one for each warp; a tile that is cut is summed by the warp
        // that begins it.
        const int t0 = first_tile(g), tiles_u = first_tile(g + 1) - t0;
        const int each = tiles_u * ra.kt / warps, more = tiles_u * ra.kt - each * warps;
        auto range = [&](int w) { return w * each + min(w, more); };
        const int tile = t0 + range(warp) / ra.kt, k_first = range(warp) - (tile - t0) * ra.kt, n_steps = each + (warp < more);
        // this warp's next item to fetch: tile ft, place fk along the row, matrix fm
        int ft = tile, fk = k_first, fm = 0, f_left = n_steps;
        auto fetch = [&]() {
            if (f_left > 0 && !dead) {
                const uint32_t slot = get & 1u;
                if (lane == 0) {
                    const uint32_t dst = codes + slot * (kItemBoxes * kBoxBytes), bar = bars + slot * 8;
                    const CUtensorMap *map = &maps.codes[kMats == 2 ? fm : 0];
                    const int y = expert * a.sh.n + ft * 16;
                    mbar_arrive_expect_tx(bar, kItemBoxes * kBoxBytes);
#pragma unroll
                    for (int i = 0; i < kItemBoxes; ++i)
                        tma_load_2d(dst + i * kBoxBytes, map, (fk * kItemBoxes + i) * 128, y, bar);
                }
                // scales: the 16-byte chunks that hold the rows' next 4 * GPB
                constexpr int kBytes = kItemBoxes * 4 * GPB;
                const uint16_t *sc = (kMats == 2 && fm ? a.m[1].scales : a.m[0].scales) + expert * a.mat_scales;
                const uint32_t sdst = scales + slot * kScales;
                if (ALIGNED) {
                    constexpr int kCp = kBytes / 16 > 0 ? kBytes / 16 : 1;   // copies of a row
                    const int r = lane / kCp, byte = lane % kCp * 16;
                    const int row = min(ft * 16 + r, a.sh.n - 1);
                    const int have = a.sh.ng * 2 - fk * kBytes - byte;
                    const uint8_t *src =
                        reinterpret_cast<const uint8_t *>(sc + int64_t(row) * a.sh.lds) + fk * kBytes + byte;
                    if (lane < 16 * kCp) {   // (zeros past the row's end)
                        if (kBytes >= 16)
                            cp16(sdst + r * kScaleRow + byte, have > 0 ? src : reinterpret_cast<const uint8_t *>(sc),
                                 max(0, min(16, have)));
                        else if (kBytes == 8)
                            cp8(sdst + r * kScaleRow, src, min(8, have));
                        else
                            cp4(sdst + r * kScaleRow, src, min(4, have));
                    }
                } else {   // rows start on any 2 bytes: from the 16 bytes before on
                    constexpr int kCp = (kBytes + 14 + 15) / 16;
                    for (int i = lane; i < 16 * kCp; i += 32) {
                        const int r = i / kCp, row = min(ft * 16 + r, a.sh.n - 1);
                        const uint8_t *first = reinterpret_cast<const uint8_t *>(sc + int64_t(row) * a.sh.lds) + fk * kBytes;
                        const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(first) & 15u);
                        const int byte = i % kCp * 16 - mis;
                        const int have = min(kBytes, a.sh.ng * 2 - fk * kBytes) - byte;
                        if (have > 0) cp16(sdst + r * kScaleRow + i % kCp * 16, first + byte, min(16, have));
                    }
                }
                ++get;
                if (++fm == kMats) {
                    fm = 0;
                    --f_left;
                    if (++fk == ra.kt) {
                        fk = 0;
                        ++ft;
                    }
                }
            }
            cp_commit();
        };
        fetch();
        fetch();
        constexpr int kSpan = 16 / GPB;   // 8-column chunks of a scale's columns
        if (MODE == MODE_MATVEC && threadIdx.x < 8) top_of[threadIdx.x] = 0u;
        int as = 0;
        if (MODE != MODE_MATVEC && threadIdx.x < cnt) as = a.perm[p0 + threadIdx.x];
        __syncthreads();   // the x rows of the unit before are no longer read
        const int n_s = x_chunks / 4;   // groups of 32
        if (MODE != MODE_MATVEC) {   // made by w4_prepare_kernel: of the token, or of the assignment
            if (threadIdx.x < cnt) {
                const int row = MODE == MODE_W12 ? as / a.topk : as;
                as_of[threadIdx.x] = as;
                row_of[threadIdx.x] = row;
                down[threadIdx.x] = a.x_down[row];
                if (MODE == MODE_W3_GROUPED) gate_of[threadIdx.x] = a.gates[as];
            }
            __syncthreads();
            for (int r = 0; r < cnt; ++r) {
                const int start_at = (r >> 1) * 4 + (r & 1);
                const uint16_t *from = a.x + int64_t(row_of[r]) * x_chunks * 8;
                const uint32_t to = smem_u32(xs) + r * ra.xstride;
                for (int c = threadIdx.x; c < x_chunks; c += threads) cp16(to + c * 16, from + c * 8, 16);
                const float *sf = a.x_starts + int64_t(row_of[r]) * n_s;
                for (int g = threadIdx.x; g < n_s / (kSpan / 4); g += threads) {
                    float o = 0.f;
                    for (int j = 0; j < kSpan / 4; ++j) o += sf[g * (kSpan / 4) + j];
                    starts[g * 16 + start_at] = starts[g * 16 + start_at + 2] = o;
                }
            }
            cp_commit();
            cp_wait<0>();
        } else {
            // the rows as they are first; each row's largest value; then in place as fp16
            // (a warp takes an even run of spans of 32 chunks, a row's part of it at a time)
            const int spans = x_chunks / 32, s0 = cnt * spans * warp / warps, s1 = cnt * spans * (warp + 1) / warps;
            auto each_row = [&](auto &&part) {
                int r = s0 / spans, b = s0 - r * spans;
                for (int left = s1 - s0; left > 0; b = 0, ++r) {
                    const int n = min(spans - b, left);
                    part(r, b * 32 + lane, n);
                    left -= n;
                }
            };
            each_row([&](int r, int c, int n) {
                const uint16_t *row = a.x + (p0 + r) * a.ldx;
#pragma unroll 4
                for (; n > 0; --n, c += 32) {
                    uint8_t *to = xs + r * ra.xstride + c * 16;
                    if (a.xvec && c * 8 + 8 <= a.sh.k)
                        cp16(smem_u32(to), row + c * 8, 16);
                    else
                        *reinterpret_cast<uint4 *>(to) = c * 8 < a.sh.k ? load8(row, c * 8, a.sh.k, false) : make_uint4(0u, 0u, 0u, 0u);
                }
            });
            cp_commit();
            cp_wait<0>();   // (each thread's own)
            each_row([&](int r, int c, int n) {
                uint32_t top = 0;
#pragma unroll 4
                for (; n > 0; --n, c += 32)
                    top = max(top, max_finite_packed(*reinterpret_cast<const uint4 *>(xs + r * ra.xstride + c * 16)));
                top = __reduce_max_sync(0xffffffffu, top);
                if (lane == 0) atomicMax(&top_of[r], top);
            });
            __syncthreads();
            each_row([&](int r, int c, int n) {
                float dn;
                const float up = scale_up(top_of[r], dn);
                if (c == 0) down[r] = dn;
#pragma unroll 4
                for (; n > 0; --n, c += 32) {
                    uint4 *p = reinterpret_cast<uint4 *>(xs + r * ra.xstride + c * 16);
                    const uint4 h = to_fragment(*p, up);
                    *p = h;
                    if (FAST) {
                        float o = offset_sum(h);
                        for (int d = 1; d < kSpan; d <<= 1) o += __shfl_xor_sync(0xffffffffu, o, d);
                        if (lane % kSpan == 0) {
                            float *to = starts + c / kSpan * 16 + (r >> 1) * 4 + (r & 1);
                            to[0] = to[2] = -o;
                        }
                    }
                }
            });
        }
        __syncthreads();
        // mma column n reads x row n (past the last one, that: nobody looks at the
        // result); this lane's products are in columns 2q and 2q + 1
        const int n = lane >> 2, q = lane & 3;
        const uint32_t xp = smem_u32(xs) + min(n, cnt - 1) * ra.xstride + q * 16;
        const uint32_t cp = smem_u32(starts) + q * 16;
        const uint32_t row_at = codes + ((lane & 8) + (lane & 7)) * 128;   // matrix lane / 8 % 2 is rows 8..
        int left = n_steps, k = k_first;
        float acc[kMats][4];
        auto write = [&](int t) {
            float most = 0.f;   // an infinity among the lane's sums (a NaN is passed over)
#pragma unroll
            for (int m = 0; m < kMats; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) most = fmaxf(most, fabsf(acc[m][i]));
            if (most == __int_as_float(0x7f800000)) {
#pragma unroll
                for (int m = 0; m < kMats; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[m][i] = settle(acc[m][i], a.m[m].scales + expert * a.mat_scales +
                                                          int64_t(min(t * 16 + n + (i >> 1) * 8, a.sh.n - 1)) * a.sh.lds, a.sh.ng);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = t * 16 + n + (i >> 1) * 8, col = 2 * q + (i & 1);
                if (col >= cnt) continue;
                const float dn = down[col];
                if (MODE == MODE_MATVEC) {
                    if (row >= a.sh.n) continue;
                    const float v = acc[0][i] * dn;
                    const int64_t y = (p0 + col) * a.ldy + row;
                    if (a.y_f32)
                        static_cast<float *>(a.y)[y] = v;
                    else
                        static_cast<__nv_bfloat16 *>(a.y)[y] = __float2bfloat16_rn(v);
                } else if (MODE == MODE_W12) {   // (features past the last one are zeros)
                    if (row < a.act_ld)
                        a.act[int64_t(as_of[col]) * a.act_ld + row] =
                            row < a.sh.n ? situ_glu_exact(acc[0][i] * dn, acc[kMats - 1][i] * dn, a.beta1, a.beta2) : 0.f;
                } else if (row < a.sh.n) {
                    a.o[int64_t(as_of[col]) * a.sh.n + row] = gate_of[col] * (acc[0][i] * dn);
                }
            }
        };
        int t = tile;
        bool whole = true;   // nothing is left in acc
        const int head_q = ra.xrows <= 4 ? 2 : 4;   // lanes of a row of acc with columns that count
        for (; left > 0; ++t) {
            const int k_from = k, k_to = min(ra.kt, k + left);
#pragma unroll
            for (int m = 0; m < kMats; ++m) acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.f;
            for (; k < k_to; ++k) {
#pragma unroll
                for (int m = 0; m < kMats; ++m) {
                    const uint32_t slot = use & 1u, bar = bars + slot * 8, phase = (use >> 1) & 1u;
                    cp_wait<1>();   // the next item's copies are one commit group
                    __syncwarp();   // the scales are copies of all lanes, and each has waited for its own only
                    if (!dead && !mbar_try_wait(bar, phase))
                        dead = !mbar_wait(bar, phase, abort_flag, err(), kWaitLimitNs);
                    if (__any_sync(0xffffffffu, dead)) {
                        dead = true;
                    } else {
                        uint32_t sp0 = scales + slot * kScales + n * kScaleRow, sp1 = sp0 + 8 * kScaleRow;
                        if (!ALIGNED) {   // where in its first 16 bytes each row starts
                            const uintptr_t sc =
                                reinterpret_cast<uintptr_t>((m ? a.m[1].scales : a.m[0].scales) + expert * a.mat_scales) +
                                k * (kItemBoxes * 4 * GPB);
                            sp0 += (sc + int64_t(min(t * 16 + n, a.sh.n - 1)) * a.sh.lds * 2) & 15u;
                            sp1 += (sc + int64_t(min(t * 16 + n + 8, a.sh.n - 1)) * a.sh.lds * 2) & 15u;
                        }
                        run_item<GPB, FAST, ALIGNED>(row_at + slot * (kItemBoxes * kBoxBytes), sp0, sp1, xp + k * (kItemCols * 2),
                                                     cp + k * (kItemBoxes * 2 * GPB * 64), a.sh.ng - k * (kItemBoxes * 2 * GPB), acc[m]);
                        ++use;
                        __syncwarp();
                        fetch();
                    }
                }
            }
            if (dead) break;
            left -= k_to - k_from;
            k = 0;
            if (k_from > 0) {   // the rest of a tile that another warp began, or a part of it
                if (q < head_q) {
#pragma unroll
                    for (int m = 0; m < kMats; ++m)
                        heads[((warp * kMats + m) * 8 + n) * head_q + q] = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
                }
            } else if (k_to < ra.kt) {   // (the range ends here)
                whole = false;
                break;
            } else {
                write(t);
            }
        }
        if (MODE == MODE_W12 && g == groups - 1) {   // tiles past the matrix only pad the activations: zeros
            for (int p = tiles + warp; p < a.tiles; p += warps) write(p);
        }
        if (tiles_u % warps) {   // (else no tile is cut)
            __syncthreads();
            if (!whole && q < head_q) {
                const int end = (t - t0 + 1) * ra.kt;   // of the tile
                for (int w = warp + 1; w < warps && range(w) < end; ++w) {
                    if (range(w) == range(w + 1)) continue;
#pragma unroll
                    for (int m = 0; m < kMats; ++m) {
                        const float4 h = heads[((w * kMats + m) * 8 + n) * head_q + q];
                        acc[m][0] += h.x;
                        acc[m][1] += h.y;
                        acc[m][2] += h.z;
                        acc[m][3] += h.w;
                    }
                }
                write(t);
            }
        }
    }
    cp_wait<0>();
    // after a wait that gave up: leave no copy in flight
    for (; use < get; ++use)
        mbar_wait(bars + (use & 1u) * 8, (use >> 1) & 1u, abort_flag, err(), kWaitLimitNs, false);
}

// Assignments grouped by expert: perm, and a list {expert, first place, rows} of the
// experts' assignments, at most `most` to an entry (entries are computed side by side).
// One block; ids outside [0, E) are left out.
__device__ __forceinline__ void group_assignments(const int32_t *idx, int n, int E, int most, int32_t *perm,
                                                  int4 *list, int32_t *n_list) {
    constexpr int kWarps = kPrepThreads / 32;
    __shared__ int cnt[kPrepThreads], s_off[kWarps], s_used[kWarps];
    const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
    cnt[e] = 0;
    __syncthreads();
    for (int i = e; i < n; i += kPrepThreads) {
        const int x = idx[i];
        if (x >= 0 && x < E) atomicAdd(&cnt[x], 1);
    }
    __syncthreads();
    // exclusive sums over the experts, of assignments and entries: within the warp, then over the warps
    const int c = cnt[e], ents = (c + most - 1) / most;
    int off = c, used = ents;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, off, d), w = __shfl_up_sync(0xffffffffu, used, d);
        if (lane >= d) {
            off += v;
            used += w;
        }
    }
    if (lane == 31) {
        s_off[warp] = off;
        s_used[warp] = used;
    }
    __syncthreads();
    int all = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
            off += s_off[w];
            used += s_used[w];
        }
        all += s_used[w];
    }
    const int first = off - c;
    for (int i = 0; i < ents; ++i) list[used - ents + i] = make_int4(e, first + i * most, min(most, c - i * most), 0);
    if (e == 0) *n_list = all;
    cnt[e] = first;   // next free place
    __syncthreads();
    // (which of an expert's assignments comes first does not matter: each is
    // computed alone)
    for (int i = e; i < n; i += kPrepThreads) {
        const int x = idx[i];
        if (x >= 0 && x < E) perm[atomicAdd(&cnt[x], 1)] = i;
    }
}

// z[t] = sum over the token's assignments of o (in order; ids outside [0, E) have none)
__global__ void __launch_bounds__(256) w4_sum_kernel(const float *__restrict__ o, const int32_t *__restrict__ idx, int k,
                                                     int E, int L, uint16_t *__restrict__ z, int64_t ldz) {
    grid_dependency_wait();
    const int64_t t = blockIdx.x;
    const int c = blockIdx.y * 256 + threadIdx.x;
    if (c >= L) return;
    float v = 0.f;
    for (int j = 0; j < k; ++j) {
        const int e = idx[t * k + j];
        if (e >= 0 && e < E) v += o[(t * k + j) * L + c];
    }
    z[t * ldz + c] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// The same sum z (idx == nullptr: o holds it, one row a token) and r = z / sqrt(mean(z^2) + eps),
// one block a token.
constexpr int kNormThreads = 512;
__global__ void __launch_bounds__(kNormThreads) w4_norm_kernel(const float *__restrict__ o, const int32_t *__restrict__ idx,
                                                               int k, int E, int L, float eps, uint16_t *__restrict__ r,
                                                               int64_t ldr) {
    grid_dependency_wait();
    extern __shared__ float zs[];   // [L]
    __shared__ float part[kNormThreads / 32];
    const int64_t t = blockIdx.x;
    float ss = 0.f;
    for (int c = threadIdx.x; c < L; c += kNormThreads) {
        float v = 0.f;
        if (idx) {
            for (int j = 0; j < k; ++j) {
                const int e = idx[t * k + j];
                if (e >= 0 && e < E) v += o[(t * k + j) * L + c];
            }
        } else {
            v = o[t * L + c];
        }
        zs[c] = v;
        ss = fmaf(v, v, ss);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = 0.f;
    for (int w = 0; w < kNormThreads / 32; ++w) ss += part[w];
    const float inv = 1.0f / sqrtf(ss / static_cast<float>(L) + eps);
    for (int c = threadIdx.x; c < L; c += kNormThreads)
        r[t * ldr + c] = __bfloat16_as_ushort(__float2bfloat16_rn(zs[c] * inv));
}

// Symmetric quantisation, one warp per row and 256 columns at a time: a lane
// has 8 columns, a group's lanes share its largest magnitude.
//   s = bf16(max|w| / 7);  u = 8 + clamp(round(w / s), -8, 7)  (8 where s is 0)
// A group with a NaN or an infinity gets that as its scale.
template <int GROUP>
__global__ void __launch_bounds__(256)
    w4_quantize_kernel(const uint16_t *__restrict__ w, int64_t rows, int k, int64_t ldw, int vec, uint8_t *__restrict__ codes,
                       int64_t ldc, int row_bytes, uint16_t *__restrict__ scales, int64_t lds, int ng) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t r = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (r >= rows) return;
    for (int c0 = 0; c0 < row_bytes * 2; c0 += 256) {
        const int c = c0 + lane * 8;
        const uint4 v = load8(w + r * ldw, c, k, vec != 0);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        float f[8], amax = 0.f;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            amax = fmaxf(amax, fabsf(f[i]));
            bad = bad || f[i] != f[i];
        }
        if (bad) amax = __int_as_float(0x7f800000);
#pragma unroll
        for (int o = GROUP / 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const __nv_bfloat16 sb = __float2bfloat16_rn(amax / 7.f);
        const float s = __bfloat162float(sb);
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            int q = 0;
            if (s > 0.f && amax < __int_as_float(0x7f800000)) q = max(-8, min(7, __float2int_rn(f[i] / s)));
            word |= uint32_t(q + 8) << (4 * i);
        }
        if (c / 2 < row_bytes) *reinterpret_cast<uint32_t *>(codes + r * ldc + c / 2) = word;
        if (c % GROUP == 0 && c / GROUP < ng) scales[r * lds + c / GROUP] = __bfloat16_as_ushort(sb);
    }
}

void make_shape(MatShape &sh, int n, int k, int group, int64_t ldc, int64_t lds, const uint16_t *const *scales,
                int n_mats, int64_t mat_scales) {
    sh.n = n;
    sh.k = k;
    sh.ldc = ldc;
    sh.lds = lds;
    sh.row_bytes = ((k + 1) / 2 + 15) / 16 * 16;
    sh.ng = (k + group - 1) / group;
    sh.kt = (k + kTaskCols - 1) / kTaskCols;
    uint64_t bits = uint64_t(lds) * 2 | uint64_t(mat_scales) * 2;
    for (int i = 0; i < n_mats; ++i) bits |= reinterpret_cast<uintptr_t>(scales[i]);
    sh.unit = bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : 2;
    sh.full = sh.unit >= 8 ? std::min(sh.row_bytes / 256, sh.ng / (kTaskCols / group)) : 0;
}

// Of a block, and every kernel's limit: the limit belongs to the kernel, so a launch that set it to its own
// size could lower it between another thread's setting and launch.
constexpr int kMaxSmem = 227 * 1024;
constexpr int kSmSmem = 228 * 1024;   // of an SM; a block takes 1 KB more than it asks for
constexpr int kExpertRows = 4;   // rows of an entry where most experts have one: they leave room for two blocks on an SM

// Warps and shared memory of a w4_kernel launch for `cols` column tasks a row tile: one warp
// per column task up to 16, and several rows of warps where there are few columns.
template <int MODE, int P>
int plan(W4Args &a, int cols, int64_t entries, int num_sms) {
    a.cols = cols;
    const int rounds = (cols + kMaxWarps - 1) / kMaxWarps;
    a.cw = (cols + rounds - 1) / rounds;
    a.rw = a.cw >= 5 ? 1 : 8 / a.cw;
    const int per = MODE == MODE_W12 ? 2 : 1;   // tiles of a unit per rt
    a.rt = std::max(1, a.rw / per);
    auto bytes = [&] { return a.cw * a.rw * kSlots * kSlotBytes + 2 * a.rt * per * a.cw * (64 * P); };
    // larger units while every SM still has four and two blocks fit on an SM
    while (a.rt * per < 8 * a.rw && entries * (a.tiles / (2 * a.rt)) >= 4 * num_sms &&
           a.cw * a.rw * kSlots * kSlotBytes + 4 * a.rt * per * a.cw * (64 * P) + 1024 <=
               kMaxSmem / (a.cw * a.rw > 8 ? 1 : P == 8 ? 2 : 3))
        a.rt *= 2;
    if (a.rw > a.rt * per) a.rw = a.rt * per;
    a.units = static_cast<int>(entries * ((a.tiles + a.rt - 1) / a.rt));
    return bytes();
}

template <int MODE, int P>
cudaError_t launch_w4(W4Args &a, int gpb, int cols, int64_t entries, int num_sms, cudaStream_t st) {
    const int smem = plan<MODE, P>(a, cols, entries, num_sms);
    const int threads = a.cw * a.rw * 32;
    auto go = [&](auto kern) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return e;
        int per_sm = 1;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, size_t(smem));
        if (e != cudaSuccess) return e;
        const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(a.units, int64_t(num_sms) * std::max(per_sm, 1)));
        return launch_kernel(kern, dim3(static_cast<unsigned>(grid)), dim3(threads), size_t(smem), st, true, a);
    };
    if (threads <= 256) {
        if (gpb == 4) return go(w4_kernel<MODE, P, 4, 256>);
        if (gpb == 2) return go(w4_kernel<MODE, P, 2, 256>);
        return go(w4_kernel<MODE, P, 1, 256>);
    }
    if (gpb == 4) return go(w4_kernel<MODE, P, 4, 512>);
    if (gpb == 2) return go(w4_kernel<MODE, P, 2, 512>);
    return go(w4_kernel<MODE, P, 1, 512>);
}

// Blocks to an SM, warps and x layout of w4_rows_kernel (matvec: one block, whose warps share the
// work of making the x rows ready); false when the x rows leave no room.
template <int MODE>
bool rows_plan(RowsArgs &ra, int k, int rows, int gpb, bool fast, bool aligned, int &blocks, int &warps, int &smem) {
    const int kt = (k + kItemCols - 1) / kItemCols;
    ra.kt = kt;
    ra.xstride = kt * kItemCols * 2 + 64;   // an odd multiple of 64 bytes: no bank conflicts between the rows
    ra.xrows = rows;
    const int fixed = rows * ra.xstride + (fast ? kt * (kItemBoxes * 2 * gpb * 64) : 0) + 160 + 16;
    // two slots and their barriers, and the sums of a tile that another warp began
    const int per_warp = 2 * (kItemBoxes * kBoxBytes + item_scales(aligned)) + 16 +
                         (MODE == MODE_W12 ? 2 : 1) * (rows <= 4 ? 256 : 512);
    blocks = kRowsPerSm;
    warps = 8;
    if (MODE == MODE_MATVEC || (fixed + 8 * per_warp + 1024) * blocks > kSmSmem) {   // one block to an SM: as many warps as fit
        blocks = 1;
        warps = std::min(8 * kRowsPerSm, (kMaxSmem - fixed) / per_warp);
    }
    smem = fixed + warps * per_warp;
    return warps >= 4;
}

// Launch of w4_rows_kernel; cudaErrorNotSupported when the x rows leave no room.
template <int MODE, bool FAST>
cudaError_t launch_rows(W4Args &a, const W4Maps &maps, int gpb, int rows, int64_t entries, int num_sms, cudaStream_t st) {
    RowsArgs ra{};
    int blocks, warps, smem;
    // whether one copy holds what an item needs of a row's scales
    const bool aligned = a.sh.unit >= std::min(16, kItemBoxes * 4 * gpb);
    if (!rows_plan<MODE>(ra, a.sh.k, rows, gpb, FAST, aligned, blocks, warps, smem)) return cudaErrorNotSupported;
    ra.a = a;
    const int tiles = (a.sh.n + 15) / 16;
    int64_t grid;
    if (MODE == MODE_MATVEC) {   // blocks to share the tiles for each 8 rows, with an item at least for each warp
        const int passes = (a.m_rows + rows - 1) / rows;
        const int64_t most = std::min<int64_t>(tiles, (int64_t(tiles) * ra.kt + warps - 1) / warps);
        grid = passes * std::max<int64_t>(1, std::min<int64_t>(most, num_sms * blocks / passes));
    } else {
        grid = std::max<int64_t>(1, std::min<int64_t>(entries * tiles, int64_t(num_sms) * blocks));
    }
    auto go = [&](auto kern) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return e;
        return launch_kernel(kern, dim3(static_cast<unsigned>(grid)), dim3(warps * 32), size_t(smem), st, true, maps, ra);
    };
    auto pick = [&](auto aligned) {
        constexpr bool A = decltype(aligned)::value;
        constexpr int kBig = 256 * kRowsPerSm;
        if (warps <= 8) {
            if (gpb == 4) return go(w4_rows_kernel<MODE, 4, FAST, A, 256>);
            if (gpb == 2) return go(w4_rows_kernel<MODE, 2, FAST, A, 256>);
            return go(w4_rows_kernel<MODE, 1, FAST, A, 256>);
        }
        if (gpb == 4) return go(w4_rows_kernel<MODE, 4, FAST, A, kBig>);
        if (gpb == 2) return go(w4_rows_kernel<MODE, 2, FAST, A, kBig>);
        return go(w4_rows_kernel<MODE, 1, FAST, A, kBig>);
    };
    return aligned ? pick(std::true_type{}) : pick(std::false_type{});
}

}  // namespace

int w4_act_ld(int inter) { return (inter + 127) / 128 * 128; }

cudaError_t launch_w4_quantize(const uint16_t *w, int64_t rows, int k, int64_t ldw, int group, uint8_t *codes,
                               int64_t ldc, uint16_t *scales, int64_t lds, cudaStream_t st) {
    const int row_bytes = ((k + 1) / 2 + 15) / 16 * 16, ng = (k + group - 1) / group;
    const int vec = ldw % 8 == 0 && reinterpret_cast<uintptr_t>(w) % 16 == 0;
    const dim3 grid(static_cast<unsigned>((rows + 7) / 8));
    auto go = [&](auto kern) {
        return launch_kernel(kern, grid, dim3(256), 0, st, true, w, rows, k, ldw, vec, codes, ldc, row_bytes, scales, lds, ng);
    };
    if (group == 32) return go(w4_quantize_kernel<32>);
    if (group == 64) return go(w4_quantize_kernel<64>);
    return go(w4_quantize_kernel<128>);
}

cudaError_t w4_status_word(unsigned **word) { return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_w4_status); }

// w4_rows_kernel starts later (the x rows first, which takes longer the more columns there are), then
// streams faster and unpacks a weight once for 8 rows.  Measured (w4_kernel | w4_rows_kernel, us):
//   1 row: 14336 x 1024 6.0 | 6.5, 3584 x 7168 9.4 | 9.0, 7168 x 7168 13.1 | 11.7, 65536 x 7168 74 | 52
//   4 rows: 3584 x 7168 10.3 | 10.7, 7168 x 7168 13.7 | 13.2, 65536 x 7168 70 | 58
//   8 rows: 3584 x 3584 9.3 | 9.0, 7168 x 3584 13.0 | 9.9, 65536 x 3584 56 | 34
//   9 rows: 512 x 7168 9.0 | 11.3, 1024 x 1024 6.6 | 5.7, 7168 x 256 7.1 | 5.1
//   32 rows: 512 x 7168 9.3 | 11.2, 2048 x 2048 9.6 | 6.7, 7168 x 3584 32 | 16
//   5 rows that start on any 2 bytes (w4_kernel reads them again for every unit):
//   1400 x 3571 8.9 | 7.9, 7001 x 3571 17.7 | 9.8
bool w4_wants_maps(int n, int k, int m, bool vec, int num_sms) {
    const int64_t tiles = (n + 15) / 16, steps = (k + kItemCols - 1) / kItemCols, passes = (m + 7) / 8;
    if (m > 4 || !vec) return tiles * passes >= 12 * steps;
    return tiles * steps >= int64_t(20) * num_sms;
}

cudaError_t launch_w4_matvec(const W4Weights &w, int n, int k, int group, const uint16_t *x, int m, int64_t ldx, void *y,
                             int64_t ldy, int y_f32, const W4Maps *maps, int num_sms, cudaStream_t st) {
    W4Args a{};
    make_shape(a.sh, n, k, group, w.ldc, w.lds, &w.scales, 1, 0);
    a.m[0] = Mat{w.codes, w.scales};
    a.x = x;
    a.ldx = ldx;
    a.m_rows = m;
    a.xvec = (m == 1 || ldx % 8 == 0) && reinterpret_cast<uintptr_t>(x) % 16 == 0;
    a.tiles = (n + 15) / 16;
    a.y = y;
    a.ldy = ldy;
    a.y_f32 = y_f32;
    if (maps) {
        const int rows = std::min(m, 8), gpb = 128 / group;
        const cudaError_t e = y_f32 ? launch_rows<MODE_MATVEC, false>(a, *maps, gpb, rows, 1, num_sms, st)
                                    : launch_rows<MODE_MATVEC, true>(a, *maps, gpb, rows, 1, num_sms, st);
        if (e != cudaErrorNotSupported) return e;
    }
    if (m <= 2) return launch_w4<MODE_MATVEC, 2>(a, 128 / group, a.sh.kt, 1, num_sms, st);
    if (m <= 4) return launch_w4<MODE_MATVEC, 4>(a, 128 / group, a.sh.kt, 1, num_sms, st);
    return launch_w4<MODE_MATVEC, 8>(a, 128 / group, a.sh.kt, (m + 7) / 8, num_sms, st);
}

size_t w4_x_bytes(int64_t rows, int k) {
    const size_t kt = (k + kItemCols - 1) / kItemCols;
    return size_t(rows) * (kt * (kItemCols * 2 + kItemCols / 8) + 4);   // rows, starts, factors
}

namespace {
// The parts of a buffer of w4_x_bytes.
void prepared(PrepArgs &r, void *buf) {
    r.xh = static_cast<uint16_t *>(buf);
    r.starts = reinterpret_cast<float *>(r.xh + int64_t(r.rows) * r.kt * kItemCols);
    r.down = r.starts + int64_t(r.rows) * r.kt * (kItemCols / 32);
}
}  // namespace

// Token by token each assignment reads its expert's weights for itself (about 0.06 us and
// 2.5 TB/s), in two launches; grouped, each expert's are read once for 8 assignments, in five
// launches.  Measured (token by token | grouped, us), experts of L x I:
//   3584 x 512, top-16: 1 token 28 | 32, 2 tokens 45 | 45; top-4: 4 tokens 29 | 31, 8 tokens 46 | 43
//   1792 x 256, top-16: 2 tokens 23 | 27, 4 tokens 37 | 35
//   1024 x 256, top-8: 8 tokens 23 | 26, 16 tokens 38 | 33; 1000 x 259, top-5: 8 tokens 18 | 23, 16 tokens 29 | 26
//   256 x 64, top-2: 64 tokens 13 | 23, 128 tokens 22 | 23, 256 tokens 37 | 25
// which the sum of bytes below, 150 KB more to an assignment, divides to within 15%.
// Rows to an entry, 4 | 8: 64 tokens of top-16 over 896 experts 335 us | 305, over 256 251 | 206,
// over 61 185 | 138; 6 tokens over 896 82 | 87 (8 rows leave room for one block on an SM).
int w4_entry_rows(const W4Experts &x) {
    const int64_t n = int64_t(x.T) * x.topk;
    if (n * (int64_t(x.L) * x.I * 3 / 2 + 150000) <= 48000000) return 0;
    auto fits = [&](int rows) {
        RowsArgs ra{};
        int blocks, warps, smem;
        return rows_plan<MODE_W12>(ra, x.L, rows, 128 / x.group, true, false, blocks, warps, smem) &&
               rows_plan<MODE_W3_GROUPED>(ra, x.I, rows, 128 / x.group, true, false, blocks, warps, smem);
    };
    if (n >= x.E && fits(8)) return 8;
    return fits(kExpertRows) ? kExpertRows : 0;
}

cudaError_t launch_w4_experts(const W4Experts &x, int num_sms, cudaStream_t st) {
    const int n = x.T * x.topk;
    const int gpb = 128 / x.group;
    W4Args b{};   // what both launches share
    b.idx = x.idx;
    b.topk = x.topk;
    b.E = x.E;
    b.list = x.list;
    b.n_list = x.n_list;
    b.perm = x.perm;
    b.gates = x.gates;
    b.act = x.act;
    b.act_ld = w4_act_ld(x.I);
    b.beta1 = x.beta1;
    b.beta2 = x.beta2;
    b.err = x.err;
    const int64_t entries = x.list ? std::min(n, std::min(n, x.E) + n / x.most) : n;
    {   // a = SiTU(W1 h) softcap(W2 h)
        W4Args a = b;
        const uint16_t *sc[2] = {x.w1.scales, x.w2.scales};
        make_shape(a.sh, x.I, x.L, x.group, x.w1.ldc, x.w1.lds, sc, 2, int64_t(x.I) * x.w1.lds);
        a.m[0] = Mat{x.w1.codes, x.w1.scales};
        a.m[1] = Mat{x.w2.codes, x.w2.scales};
        a.mat_codes = int64_t(x.I) * x.w1.ldc;
        a.mat_scales = int64_t(x.I) * x.w1.lds;
        a.x = x.h;
        a.ldx = x.ldh;
        a.xvec = x.ldh % 8 == 0 && reinterpret_cast<uintptr_t>(x.h) % 16 == 0;
        a.tiles = b.act_ld / 16;
        cudaError_t e;
        if (x.list) {
            PrepArgs r{};
            r.x = x.h;
            r.ldx = x.ldh;
            r.rows = x.T;
            r.k = x.L;
            r.vec = a.xvec;
            r.kt = (x.L + kItemCols - 1) / kItemCols;
            prepared(r, x.xbuf);
            r.idx = x.idx;
            r.n = n;
            r.E = x.E;
            r.perm = x.perm;
            r.most = x.most;
            r.list = x.list;
            r.n_list = x.n_list;
            e = launch_kernel(w4_prepare_kernel<false, kPrepThreads>, dim3(static_cast<unsigned>(x.T + 1)), dim3(kPrepThreads), 0,
                              st, true, r);
            if (e != cudaSuccess) return e;
            W4Args b2 = a;
            b2.x = r.xh;
            b2.x_starts = r.starts;
            b2.x_down = r.down;
            e = launch_rows<MODE_W12, true>(b2, x.maps12, gpb, x.most, entries, num_sms, st);
        } else {
            e = launch_w4<MODE_W12, 2>(a, gpb, a.sh.kt, entries, num_sms, st);
        }
        if (e != cudaSuccess) return e;
    }
    W4Args a = b;
    make_shape(a.sh, x.L, x.I, x.group, x.w3.ldc, x.w3.lds, &x.w3.scales, 1, int64_t(x.L) * x.w3.lds);
    a.m[0] = Mat{x.w3.codes, x.w3.scales};
    a.mat_codes = int64_t(x.L) * x.w3.ldc;
    a.mat_scales = int64_t(x.L) * x.w3.lds;
    a.tiles = (x.L + 15) / 16;
    if (!x.list) {   // z by token
        a.y = x.norm ? static_cast<void *>(x.zf) : x.z;
        a.ldy = x.norm ? x.L : x.ldz;
        a.y_f32 = x.norm;
        const cudaError_t e = launch_w4<MODE_W3_TOKEN, 2>(a, gpb, x.topk * a.sh.kt, x.T, num_sms, st);
        if (e != cudaSuccess || !x.norm) return e;
        return launch_kernel(w4_norm_kernel, dim3(static_cast<unsigned>(x.T)), dim3(kNormThreads), size_t(x.L) * 4, st, true,
                             static_cast<const float *>(x.zf), static_cast<const int32_t *>(nullptr), 1, 1, x.L, x.rms_eps, x.z,
                             x.ldz);
    }
    a.o = x.o;
    PrepArgs r{};
    r.act = x.act;
    r.ldx = r.k = b.act_ld;
    r.rows = n;
    r.kt = (x.I + kItemCols - 1) / kItemCols;
    prepared(r, x.xbuf3);
    r.idx = x.idx;
    r.E = x.E;
    cudaError_t e = launch_kernel(w4_prepare_kernel<true, 64>, dim3(static_cast<unsigned>(n)), dim3(64), 0, st, true, r);
    if (e != cudaSuccess) return e;
    a.x = r.xh;
    a.x_starts = r.starts;
    a.x_down = r.down;
    e = launch_rows<MODE_W3_GROUPED, true>(a, x.maps3, gpb, x.most, entries, num_sms, st);
    if (e != cudaSuccess) return e;
    if (x.norm)
        return launch_kernel(w4_norm_kernel, dim3(static_cast<unsigned>(x.T)), dim3(kNormThreads), size_t(x.L) * 4, st, true, x.o,
                             x.idx, x.topk, x.E, x.L, x.rms_eps, x.z, x.ldz);
    return launch_kernel(w4_sum_kernel, dim3(static_cast<unsigned>(x.T), static_cast<unsigned>((x.L + 255) / 256)),
                         dim3(256), 0, st, true, x.o, x.idx, x.topk, x.E, x.L, x.z, x.ldz);
}

}  // namespace lmoe
