// qg_w8a8.hip -- matrix product in 8-bit integers.
//
//   y[t][n] = (sum_k xq[t][k] w[n][k]) * dx[t] * dw[n],  dx[t] = amax_k |x[t][k]| / 127,
//   xq = rint(x / dx).
//
// The sums are exact in 32-bit integers (K <= 2^17), so no order of summation changes a result.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "qg_device.hpp"
#include "qg_internal.hpp"

namespace qg {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

constexpr float kPer127 = 1.0f / 127.0f;

__device__ __forceinline__ uint32_t code8(float x) {
    const float r = __builtin_rintf(x);
    return (uint32_t)(int)__builtin_amdgcn_fmed3f(r, -127.f, 127.f) & 0xffu;
}

// A row's scale from the largest |x| as bits; an infinity makes the row NaN as a whole.
__device__ __forceinline__ float row_scale(uint32_t top) {
    return top >= 0x7f800000u ? __builtin_nanf("") : __uint_as_float(top) * kPer127;
}

// 8 values as 8 code bytes.
__device__ __forceinline__ uint2 code8x8(const float (&v)[8], float inv) {
    uint32_t w[2];
#pragma unroll
    for (int e = 0; e < 2; e++)
        w[e] = code8(v[4 * e] * inv) | code8(v[4 * e + 1] * inv) << 8 | code8(v[4 * e + 2] * inv) << 16 |
               code8(v[4 * e + 3] * inv) << 24;
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float inverse(float d) { return d > 0.f ? fminf(1.0f / d, 3.402823466e+38f) : 0.f; }

__device__ __forceinline__ uint32_t max8(const float (&v)[8], uint32_t top) {
#pragma unroll
    for (int e = 0; e < 8; e++) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
    return top;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    return v;
}

// One workgroup codes one row of X, held in registers up to K = 16384 (longer rows are read again for
// their codes).  K % 16 == 0.
template <int XT>
__global__ __launch_bounds__(512) void x_code_kernel(const void* X, int K, int8_t* codes, float* scales) {
    constexpr int kHeld = 4;
    __shared__ uint32_t sh[8];
    const int64_t base = (int64_t)blockIdx.x * K;
    float v[kHeld][8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kHeld; i++) {
        const int k = 8 * threadIdx.x + 4096 * i;
        if (k < K) {
            x_load8<XT>(X, base + k, v[i]);
            top = max8(v[i], top);
        }
    }
    for (int k = 8 * threadIdx.x + 4096 * kHeld; k < K; k += 4096) {
        float x[8];
        x_load8<XT>(X, base + k, x);
        top = max8(x, top);
    }
    top = wave_max(top);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; w++) top = max(top, sh[w]);
    const float d = row_scale(top), inv = inverse(d);
    if (threadIdx.x == 0) scales[blockIdx.x] = d;
#pragma unroll
    for (int i = 0; i < kHeld; i++) {
        const int k = 8 * threadIdx.x + 4096 * i;
        if (k < K) *(uint2*)(codes + base + k) = code8x8(v[i], inv);
    }
    for (int k = 8 * threadIdx.x + 4096 * kHeld; k < K; k += 4096) {
        float x[8];
        x_load8<XT>(X, base + k, x);
        *(uint2*)(codes + base + k) = code8x8(x, inv);
    }
}

template <int YT>
__device__ __forceinline__ void store_y(void* Y, int64_t i, float v) {
    if constexpr (YT == XT_F32)
        ((float*)Y)[i] = v;
    else
        ((uint16_t*)Y)[i] = f32_to_16<YT>(keep_f32(v));
}
__device__ __forceinline__ void store_any(void* Y, int yt, int64_t i, float v) {
    if (yt == XT_F32)
        store_y<XT_F32>(Y, i, v);
    else if (yt == XT_F16)
        store_y<XT_F16>(Y, i, v);
    else
        store_y<XT_BF16>(Y, i, v);
}

// ---- few tokens: the weights stream once -----------------------------------------------------------
// A workgroup of KS wavefronts takes 16 RN weight rows and all (at most 16 TT) tokens; the wavefronts
// take 128-byte pieces of K in turn and their integer sums are joined at the end.  A wavefront copies its
// pieces of both operands straight into its own part of shared memory, AHEAD of them on their way, 8 rows
// of whole 128-byte lines a copy: loads into registers in the operands' layout (16 rows of 64 bytes) are
// bound by the lines that a load touches.  A row's 16-byte chunks lie at slot chunk ^ (row / 2 % 8), so
// that reads meet all banks.  CODES > 0 (few codes): every workgroup codes X itself into CODES bytes of
// shared memory while its first weights are on their way, which saves a launch.
// Bound by memory: one token 4096 x 4096 5.5 us (3.0 TB/s of 16.8 MB), 45
// tokens 11009 x 4112 13 us after the 2.4-4 us in which X is coded (3.5 TB/s).
constexpr int kFusedCodes = 32768, kFusedLds = 34 << 10;  // X codes a workgroup keeps (fewer than), bytes with pitches

__host__ __device__ __forceinline__ int fused_pitch(int K) { return (K + 127) / 128 * 128 + 16; }

// The KS wavefronts share the rows out evenly (one row: all on it); a wavefront's part of a row stays in
// registers up to 4096 values.
template <int XT, int KS>
__device__ __forceinline__ void code_rows_lds(const void* X, int K, int T, int8_t* xs, float* dx, uint32_t* part) {
    constexpr int kHeld = 8;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), pitch = fused_pitch(K);
    const int split = T <= 1 ? KS : T <= 2 ? KS / 2 : T <= 4 ? KS / 4 : KS >= 8 ? KS / 8 : 1;  // wavefronts a row
    const int rows = KS / split;                                                              // rows at a time
    for (int t0 = 0; t0 < T; t0 += rows) {
        const int t = t0 + wave / split, sub = wave % split;
        const int64_t base = (int64_t)min(t, T - 1) * K;
        const int k0 = 8 * (64 * sub + lane), step = 512 * split;
        float v[kHeld][8];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kHeld; i++) {
            if (512 * sub + step * i >= K) break;
            const int k = k0 + step * i;
#pragma unroll
            for (int e = 0; e < 8; e++) v[i][e] = 0.f;
            if (k < K) x_load8<XT>(X, base + k, v[i]);
            top = max8(v[i], top);
        }
        for (int k = k0 + step * kHeld; k < K; k += step) {
            float x[8];
            x_load8<XT>(X, base + k, x);
            top = max8(x, top);
        }
        top = wave_max(top);
        if (lane == 0) part[wave] = top;
        __syncthreads();
        for (int w = 0; w < split; w++) top = max(top, part[wave / split * split + w]);
        const float d = row_scale(top), inv = inverse(d);
        if (t < T) {
            if (lane == 0 && sub == 0) dx[t] = d;
#pragma unroll
            for (int i = 0; i < kHeld; i++) {
                if (512 * sub + step * i >= K) break;
                const int k = k0 + step * i;
                if (k < pitch - 16) *(uint2*)(xs + t * pitch + k) = code8x8(v[i], inv);
            }
            for (int k = k0 + step * kHeld; k < pitch - 16; k += step) {
                float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (k < K) x_load8<XT>(X, base + k, x);
                *(uint2*)(xs + t * pitch + k) = code8x8(x, inv);
            }
        }
        __syncthreads();
    }
}

template <int TT, int RN, int KS, int AHEAD, int CODES>
__global__ __launch_bounds__(64 * KS) void w8a8_rows_kernel(W8A8Params p) {
    constexpr bool FUSED = CODES > 0;
    constexpr int RP = 16 * RN + 4;                    // pitch of the sums
    constexpr int kPiece = (RN + (FUSED ? 0 : TT)) * 2048, kRing = KS * kPiece;
    static_assert(AHEAD == 1 || AHEAD == 2, "ring");
    constexpr int kRed = KS * 16 * TT * RP * 4;
    // one array a place in the ring, so that a read of one never waits for copies into another
    __shared__ __attribute__((aligned(16))) int8_t s0[kRing > kRed ? kRing : kRed];
    __shared__ __attribute__((aligned(16))) int8_t s1[AHEAD > 1 ? kRing : 16];
    __shared__ __attribute__((aligned(16))) int8_t codes[FUSED ? CODES : 16];
    __shared__ float dx[16];
    __shared__ uint32_t part[KS];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * RN, K = p.K;
    // this split's pieces
    const int lo = blockIdx.y * p.per, units = min(lo + p.per, (K + 127) / 128), end = min(K, 128 * units);
    const int pitch = fused_pitch(K);
    const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc((void*)(p.w + (int64_t)n0 * K), 0,
                                                                        min(16 * RN, p.N - n0) * K, 0x00020000);
    const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc((void*)p.xq, 0, FUSED ? 0 : p.T * K, 0x00020000);
    // The sums are integers, so each workgroup begins at a piece of its own: begun together at the rows'
    // starts, workgroups meet on the same memory channels where K is a power of two (16 tokens 8192 x 8192:
    // 21.9 us so, 16.3 us with pieces 5 apart; one token, coded here, 8192 x 4096 10.2 and 8.6 us).  The least form, one
    // workgroup a CU, has more of beginning at once (one token 4096 x 1024 4.5 us so, 4.8 us with pieces apart).
    constexpr bool kApart = !FUSED || RN > 1;
    const int count = units - lo, first = kApart ? (int)(5 * blockIdx.x % (unsigned)max(count, 1)) : 0;
    auto piece = [&](int u) {
        const int v = u + first;
        return !kApart ? u : u >= units ? 0x400000 : v >= units ? v - count : v;
    };
    // copy i has rows 8 i .. 8 i + 7
    const int even = 16 * ((lane & 7) ^ (lane >> 4)), odd = even ^ 64, from = (lane >> 3) * K;
    auto copy = [&](int8_t* s, int nth) {
        const int u = piece(nth);
        const int at[2] = {128 * u + even < end ? from + even + 128 * u : 0x40000000,
                           128 * u + odd < end ? from + odd + 128 * u : 0x40000000};
        int8_t* to = s + wave * kPiece;
#pragma unroll
        for (int i = 0; i < 2 * RN; i++) buffer_copy16_lds(wr, to + i * 1024, at[i & 1] + 8 * i * K);
        if constexpr (!FUSED) {
#pragma unroll
            for (int i = 0; i < 2 * TT; i++) buffer_copy16_lds(xr, to + (2 * RN + i) * 1024, at[i & 1] + 8 * i * K);
        }
    };
    i32x4_t acc[RN][TT] = {};
    auto multiply = [&](const int8_t* s, int nth) {
        const int u = piece(nth);
        const int8_t* at = s + wave * kPiece + r * 128;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int slot = 16 * ((4 * h + g) ^ (lane >> 1 & 7));
            i32x4_t w[RN], x[TT];
#pragma unroll
            for (int i = 0; i < RN; i++) w[i] = *(const i32x4_t*)(at + i * 2048 + slot);
#pragma unroll
            for (int t = 0; t < TT; t++) {
                if constexpr (FUSED)
                    x[t] = *(const i32x4_t*)(codes + min(16 * t + r, p.T - 1) * pitch + (u < units ? 128 * u + 64 * h + 16 * g : 0));
                else
                    x[t] = *(const i32x4_t*)(at + (RN + t) * 2048 + slot);
            }
#pragma unroll
            for (int t = 0; t < TT; t++)
#pragma unroll
                for (int i = 0; i < RN; i++) acc[i][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[i], x[t], acc[i][t], 0, 0, 0);
        }
    };
    copy(s0, lo + wave);
    if constexpr (AHEAD > 1) copy(s1, lo + wave + KS);
    if constexpr (FUSED) {
        if (p.xt == XT_F32)
            code_rows_lds<XT_F32, KS>(p.X, K, p.T, codes, dx, part);
        else if (p.xt == XT_F16)
            code_rows_lds<XT_F16, KS>(p.X, K, p.T, codes, dx, part);
        else
            code_rows_lds<XT_BF16, KS>(p.X, K, p.T, codes, dx, part);
    }
    // a wavefront keeps to its own pieces, so nothing is waited for but its own copies; a place is copied
    // to again only when what was read from it has arrived
    constexpr int kYounger = (AHEAD - 1) * 2 * (RN + (FUSED ? 0 : TT));  // copies after the piece's own
    static_assert(kYounger < 64, "ring");
    auto turn = [&](int8_t* s, int u) {
        __builtin_amdgcn_s_waitcnt(0x0f70 | (kYounger & 15) | (kYounger >> 4) << 14);
        __builtin_amdgcn_sched_barrier(0);
        multiply(s, u);
        __builtin_amdgcn_s_waitcnt(0xc07f);
        __builtin_amdgcn_sched_barrier(0);
        copy(s, u + KS * AHEAD);
    };
    for (int u0 = lo + wave; u0 < units; u0 += KS * AHEAD) {
        turn(s0, u0);
        if constexpr (AHEAD > 1) turn(s1, u0 + KS);
    }
    __builtin_amdgcn_s_waitcnt(0x0f70);  // the last copies have landed before their place is used again
    __syncthreads();
    int* red = (int*)s0;
#pragma unroll
    for (int i = 0; i < RN; i++)
#pragma unroll
        for (int t = 0; t < TT; t++)
            *(i32x4_t*)(red + (wave * 16 * TT + 16 * t + r) * RP + 16 * i + 4 * g) = acc[i][t];
    __syncthreads();
    for (int x = threadIdx.x; x < 16 * TT * 16 * RN; x += 64 * KS) {
        const int t = x / (16 * RN), n = x % (16 * RN);
        if (t >= p.T || n0 + n >= p.N) continue;
        int sum = 0;
#pragma unroll
        for (int v = 0; v < KS; v++) sum += red[(v * 16 * TT + t) * RP + n];
        if (!FUSED && p.splits > 1) {
            p.part[((int64_t)blockIdx.y * p.T + t) * p.N + n0 + n] = sum;
            continue;
        }
        const float d = FUSED ? dx[t] : p.xs[t];
        store_any(p.Y, p.yt, (int64_t)t * p.N + n0 + n, (float)sum * d * p.ws[n0 + n]);
    }
}

// ---- many tokens: tiles ----------------------------------------------------------------------------
// A workgroup takes BT tokens x BN weight rows; both operands pass through shared memory in stages of
// 128 k, copied straight from memory while the R - 1 stages before are multiplied.  A row's 16-byte chunks
// lie at slot chunk ^ (row / 2 % 8): the 16 lanes that are read at a time meet all 64 banks (with
// chunk ^ (row % 8) every bank met two of them: 22 % of the kernel's cycles).  The one barrier of a stage
// stands before its last products: by then every wavefront holds their operands, so the stage's place is
// free for the copies of the stage after next, and the next stage's first operands are read during them.
// 8192^3: 450 us and 36 us for X's codes, 2.27 POP/s with them (a library's product in 8-bit integers of the
// same size: 514 us without coding); 66 % of the cycles are products, and the clock falls to 1.5-1.8 GHz under
// them: bound by power.
template <int N>
struct Frags {
    i32x4_t f[N];
};

template <int MT, int NT, int WT, int WN, int R>
__global__ __launch_bounds__(64 * WT * WN) void w8a8_tile_kernel(W8A8Params p, int tiles_t, int tiles_n) {
    constexpr int BT = 32 * MT * WT, BN = 32 * NT * WN, NW = WT * WN;
    constexpr int XC = BT / 8 / NW, WC = BN / 8 / NW;  // copies of 8 rows a wavefront and stage
    static_assert(XC * 8 * NW == BT && WC * 8 * NW == BN && NT % 2 == 0 && NW * 8192 <= (BT + BN) * 128, "tile");
    __shared__ __attribute__((aligned(16))) int8_t s0[(BT + BN) * 128];
    __shared__ __attribute__((aligned(16))) int8_t s1[(BT + BN) * 128];
    __shared__ __attribute__((aligned(16))) int8_t s2[R > 2 ? (BT + BN) * 128 : 16];
    __shared__ __attribute__((aligned(16))) int8_t s3[R > 2 ? (BT + BN) * 128 : 16];
    const int lane = threadIdx.x & 63, r = lane & 31, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wt = wave % WT, wn = wave / WT;

    // consecutive workgroups go to the 8 dies in turn: each die gets a run of tiles, in patches of 4
    // token tiles, so that its cache holds the operands its workgroups share
    const int total = tiles_t * tiles_n, per = total / 8, rem = total % 8, die = blockIdx.x & 7;
    int lin = die * per + min(die, rem) + (blockIdx.x >> 3);
    const int width = 4 * tiles_n, first = lin / width * 4, tall = min(tiles_t - first, 4);
    lin %= width;
    const int t0 = (first + lin % tall) * BT, n0 = lin / tall * BN;

    const int K = p.K;
    const int lo = blockIdx.y * p.per, stages = min(lo + p.per, (K + 127) / 128), end = min(K, 128 * stages);
    const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc((void*)(p.xq + (int64_t)t0 * K), 0,
                                                                        min(BT, p.T - t0) * K, 0x00020000);
    const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc((void*)(p.w + (int64_t)n0 * K), 0,
                                                                        min(BN, p.N - n0) * K, 0x00020000);
    const int chunk = (lane & 7) ^ ((lane >> 4) + 4 * (wave & 1));  // of the row, for this lane's slot
    const int voff = (8 * wave + (lane >> 3)) * K + 16 * chunk;
    auto copy = [&](int st, int8_t* s) {
        const int k = 128 * st + 16 * chunk < end ? voff + 128 * st : 0x40000000;  // past the end: zeros
#pragma unroll
        for (int i = 0; i < XC; i++) buffer_copy16_lds(xr, s + (i * NW + wave) * 1024, k + i * NW * 8 * K);
#pragma unroll
        for (int i = 0; i < WC; i++) buffer_copy16_lds(wr, s + BT * 128 + (i * NW + wave) * 1024, k + i * NW * 8 * K);
    };
    i32x16_t acc[NT][MT] = {};
    const int xrow = (32 * MT * wt + r) * 128, wrow = (BT + 32 * NT * wn + r) * 128;
    auto frags = [&](const int8_t* s, int j, Frags<MT>& x, Frags<NT>& w) {
        const int slot = 16 * ((2 * j + g) ^ (lane >> 1 & 7));
#pragma unroll
        for (int i = 0; i < MT; i++) x.f[i] = *(const i32x4_t*)(s + xrow + i * 4096 + slot);
#pragma unroll
        for (int i = 0; i < NT; i++) w.f[i] = *(const i32x4_t*)(s + wrow + i * 4096 + slot);
    };
    Frags<MT> x[2];
    Frags<NT> w[2];
    auto multiply = [&](int j) {
#pragma unroll
        for (int a = 0; a < NT; a++)
#pragma unroll
            for (int b = 0; b < MT; b++)
                acc[a][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[j].f[a], x[j].f[b], acc[a][b], 0, 0, 0);
        // the next step's reads go between this step's products, and no further ahead
#pragma unroll
        for (int i = 0; i < MT + NT; i++) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int kYounger = (R - 2) * (XC + WC);  // copies of later stages than the next
    static_assert((R == 2 || R == 4) && kYounger < 64, "ring");
    auto stage = [&](int st, int8_t* s, const int8_t* next) {
#pragma unroll
        for (int j = 0; j < 3; j++) {
            frags(s, j + 1, x[(j + 1) & 1], w[(j + 1) & 1]);
            multiply(j & 1);
        }
        // own copies of the next stage have landed, own reads have arrived
        __builtin_amdgcn_s_waitcnt(0x0070 | (kYounger & 15) | (kYounger >> 4) << 14);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        copy(st + R, s);
        __builtin_amdgcn_sched_barrier(0);
        frags(next, 0, x[0], w[0]);
        multiply(1);
    };
    // two arrays, so that a read of one never waits for the copies into the other; past the last stage the
    // copies are zeros
    copy(lo, s0);
    copy(lo + 1, s1);
    if constexpr (R > 2) {
        copy(lo + 2, s2);
        copy(lo + 3, s3);
    }
    __syncthreads();
    frags(s0, 0, x[0], w[0]);
    __builtin_amdgcn_sched_barrier(0);
    for (int st = lo; st < stages; st += R) {
        stage(st, s0, s1);
        stage(st + 1, s1, R > 2 ? s2 : s0);
        if constexpr (R > 2) {
            if (st + 2 >= stages) break;
            stage(st + 2, s2, s3);
            stage(st + 3, s3, s0);
        }
    }
    __builtin_amdgcn_s_waitcnt(0x0f70);  // the last copy has landed before its place is used again
    __syncthreads();

    if (p.splits > 1) {
#pragma unroll
        for (int b = 0; b < MT; b++) {
            const int t = t0 + 32 * (MT * wt + b) + r;
            if (t >= p.T) continue;
            int* to = p.part + ((int64_t)blockIdx.y * p.T + t) * p.N;
#pragma unroll
            for (int a = 0; a < NT; a++)
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    const int n = n0 + 32 * (NT * wn + a) + 8 * (e >> 2) + 4 * g + (e & 3);
                    if (n < p.N) to[n] = acc[a][b][e];
                }
        }
        return;
    }

    // 32 tokens x 64 rows at a time through this wavefront's 8 KiB, so that stores are whole lines
    float* out = (float*)(s0 + wave * 8192);
    const bool wide = p.N % 8 == 0 && ((uintptr_t)p.Y & 15) == 0;
#pragma unroll
    for (int b = 0; b < MT; b++) {
        const int tb = t0 + 32 * (MT * wt + b);
        const float d = p.xs[min(tb + r, p.T - 1)];
#pragma unroll
        for (int a = 0; a < NT; a += 2) {
            const int nb = n0 + 32 * (NT * wn + a);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const i32x16_t& c = acc[a + (i >> 2)][b];
                const int q = 4 * (i & 3);
                f32x4_t v = {(float)c[q] * d, (float)c[q + 1] * d, (float)c[q + 2] * d, (float)c[q + 3] * d};
                const int at = 2 * i + g;  // which four of the 64 rows
                *(f32x4_t*)(out + r * 64 + 4 * (at ^ (r & 15))) = v;
            }
            __builtin_amdgcn_wave_barrier();
            if (wide && p.yt != XT_F32) {
                const int n = nb + 8 * (lane & 7);
                float s[8];
#pragma unroll
                for (int e = 0; e < 8; e++) s[e] = p.ws[min(n + e, p.N - 1)];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int t = 8 * i + (lane >> 3);
                    const f32x4_t lo = *(const f32x4_t*)(out + t * 64 + 4 * ((2 * (lane & 7)) ^ (t & 15)));
                    const f32x4_t hi = *(const f32x4_t*)(out + t * 64 + 4 * ((2 * (lane & 7) + 1) ^ (t & 15)));
                    if (tb + t >= p.T || n >= p.N) continue;
                    uint32_t y[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const float u = keep_f32((e < 2 ? lo[2 * e] : hi[2 * e - 4]) * s[2 * e]);
                        const float v = keep_f32((e < 2 ? lo[2 * e + 1] : hi[2 * e - 3]) * s[2 * e + 1]);
                        y[e] = p.yt == XT_F16 ? (uint32_t)f32_to_f16_bits(u) | (uint32_t)f32_to_f16_bits(v) << 16
                                              : (uint32_t)f32_to_bf16_bits(u) | (uint32_t)f32_to_bf16_bits(v) << 16;
                    }
                    *(uint4*)((uint16_t*)p.Y + (int64_t)(tb + t) * p.N + n) = make_uint4(y[0], y[1], y[2], y[3]);
                }
            } else {
                const int n = nb + lane;
                const float s = p.ws[min(n, p.N - 1)];
                for (int t = 0; t < 32 && tb + t < p.T; t++) {
                    const float v = out[t * 64 + 4 * ((lane >> 2) ^ (t & 15)) + (lane & 3)];
                    if (n < p.N) store_any(p.Y, p.yt, (int64_t)(tb + t) * p.N + n, v * s);
                }
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
}

// The sums of the splits of K; they are integers, so their order does not matter.
__global__ __launch_bounds__(256) void w8a8_join_kernel(W8A8Params p) {
    const int n = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
    if (n >= p.N) return;
    const int64_t all = (int64_t)p.T * p.N, at = (int64_t)t * p.N + n;
    int sum = 0;
#pragma unroll 8
    for (int i = 0; i < p.splits; i++) sum += p.part[i * all + at];
    store_any(p.Y, p.yt, at, (float)sum * p.xs[t] * p.ws[n]);
}

// The streaming kernel and the tiles, us: 72, 96 tokens 11000 x 4112 21.8, 23.5 and 24.5, 24.3, 14336 x 4096 25.6,
// 27.2 and 21.3, 22.5, 28672 x 8192 77, 80 and 63, 65; 128 tokens 4096 x 14336 39 and 44-47, 6144 x 4096 20.8 and
// 16.1, 20000 x 2048 35 and 21.
bool streams(int N, int T) { return T <= 64 || (T <= 96 && N <= 12288) || (T <= 128 && N <= 5120); }
// Coding X in every workgroup saves a launch (2.5 us) but is paid again by every workgroup that a CU gets and
// grows with X.  One launch and two, us: 4096 x 4096, 1, 4, 8 tokens 6.3, 7.3, 8.6 and 7.9, 8.1, 8.0; 2048 x 8192,
// 1, 4 tokens 6.9, 9.0 and 8.0, 8.2; 4096 x 14336, 1, 2, 4 tokens 12.5, 14.2, 16.2 and 14.0, 15.3, 14.0; with two
// row blocks a workgroup 8192 x 2048, 1, 4 tokens 6.1, 6.8 and 8.1, 8.2; 8192 x 4096, 1, 2, 4, 8 tokens 8.5, 9.1,
// 10.1, 12.2 and 9.8; past that it loses: 20000 x 2048, 1, 8 tokens 14.2, 18.7 and 12.3, 12.8.
constexpr int kFusedRows = 4096;
bool fused(int N, int K, int T) {
    return T <= 8 && N <= 2 * kFusedRows && (int64_t)T * K * (N <= kFusedRows ? 1 : 2) < kFusedCodes;
}
static_assert(kFusedCodes + 8 * (127 + 16) <= kFusedLds, "codes");

template <int TT, int RN, int KS, int CODES>
void launch_rows(const W8A8Params& p, hipStream_t s) {
    constexpr int kRing = KS * (RN + (CODES ? 0 : TT)) * 2048, kRed = KS * 16 * TT * (16 * RN + 4) * 4;
    constexpr int AHEAD = (kRed > kRing ? kRed : kRing) + kRing + CODES + 2048 <= 160 << 10 ? 2 : 1;
    w8a8_rows_kernel<TT, RN, KS, AHEAD, CODES><<<dim3((p.N + 16 * RN - 1) / (16 * RN), p.splits), 64 * KS, 0, s>>>(p);
}

// Weight rows a workgroup: the fullest CU reads (16 RN + 16 TT) rows for each workgroup that it gets, and
// that bounds the kernel (45 tokens, 11009 x 4112: RN 1, 2, 3, 4: 28.8, 26.1, 21.5, 23.2 us).
int rows_of(int N, int TT) {
    int best = 1;
    int64_t least = 0;
    for (int rn = 1; rn <= 4; rn++) {
        const int64_t groups = (N + 16 * rn - 1) / (16 * rn), cost = (groups + 255) / 256 * (rn + TT);
        if (rn == 1 || cost < least) best = rn, least = cost;
    }
    return best;
}

template <int TT, int KS>
void launch_few(const W8A8Params& p, hipStream_t s) {
    switch (rows_of(p.N, TT)) {
        case 1: return launch_rows<TT, 1, KS, 0>(p, s);
        case 2: return launch_rows<TT, 2, KS, 0>(p, s);
        case 3: return launch_rows<TT, 3, KS, 0>(p, s);
        default: return launch_rows<TT, 4, KS, 0>(p, s);
    }
}

template <int MT, int NT, int WT, int WN, int R>
void launch_tile(const W8A8Params& p, hipStream_t s) {
    const int tt = (p.T + 32 * MT * WT - 1) / (32 * MT * WT), tn = (p.N + 32 * NT * WN - 1) / (32 * NT * WN);
    w8a8_tile_kernel<MT, NT, WT, WN, R><<<dim3(tt * tn, p.splits), 64 * WT * WN, 0, s>>>(p, tt, tn);
}

}  // namespace

namespace {
int64_t tiles_of(int N, int T, int side) { return (int64_t)((T + side - 1) / side) * ((N + side - 1) / side); }

// Tiles of 256 a side: a CU takes one in the time of 4/3 of two tiles of 128 (768 tokens 14336 x 4096: 62 and 77
// us; 1024 tokens 8192 x 8192: 106 and 84 us).  Tiles of 128: a CU holds two of them with two stages each, or one
// with four, which is the faster where there are no more than CUs (384 tokens 14336 x 4096: 42 and 55 us; 256
// tokens: 37 and 31 us).
bool large_tiles(int N, int T) {
    return 4 * ((tiles_of(N, T, 256) + 255) / 256) < 3 * ((tiles_of(N, T, 128) + 511) / 512);
}

// Tokens of the streaming kernel's form that a call takes, by 16.
int tokens_of(int T) {
    const int tt = (T + 15) / 16;
    return tt <= 4 ? tt : tt <= 6 ? 6 : 8;
}

// Splits of K over workgroups, where there are few of them for long rows: their sums take a third launch
// (131 tokens, 315 x 8896: 30 us in one, 15 us in eight), which few tokens do not repay (1024 x 8192, 16, 32, 64,
// 96 tokens 8.5, 10.2, 12.8, 15.6 us in one, 10.4, 10.5, 11.5, 12.9 us in four; 2048 x 8192, 32, 64, 128 tokens
// 10.4, 12.9, 19.7 us in one, 11.1, 12.5, 16.7 us in two).
void set_splits(W8A8Params& p) {
    const int pieces = (p.K + 127) / 128;
    int64_t groups, least;
    if (streams(p.N, p.T)) {
        const int tt = tokens_of(p.T), rn = rows_of(p.N, tt);
        groups = (p.N + 16 * rn - 1) / (16 * rn), least = 16;
        if (pieces * (rn + tt) < 256) groups = 256;
    } else {
        groups = tiles_of(p.N, p.T, 128) > 160 ? 256 : tiles_of(p.N, p.T, 64), least = 8;
    }
    p.splits = 1;
    p.per = pieces;
    if (fused(p.N, p.K, p.T) || groups > 128 || pieces < 3 * least) return;
    const int64_t splits = std::min(256 / groups, pieces / least);
    p.per = (int)((pieces + splits - 1) / splits + 3) / 4 * 4;
    p.splits = (pieces + p.per - 1) / p.per;
}

size_t codes_bytes(int K, int T) { return ((size_t)T * K + 255) / 256 * 256 + ((size_t)T * 4 + 255) / 256 * 256; }
}  // namespace

size_t w8a8_workspace(int N, int K, int T) {
    if (fused(N, K, T)) return 0;
    W8A8Params p{};
    p.N = N, p.K = K, p.T = T;
    set_splits(p);
    return codes_bytes(K, T) + (p.splits > 1 ? (size_t)p.splits * T * N * 4 : 0);
}

hipError_t launch_w8a8(W8A8Params p, void* ws, hipStream_t s) {
    const bool fuse = fused(p.N, p.K, p.T);
    set_splits(p);
    if (!fuse) {
        float* xs = (float*)((char*)ws + ((size_t)p.T * p.K + 255) / 256 * 256);
        int8_t* xq = (int8_t*)ws;
        p.xq = xq;
        p.xs = xs;
        p.part = (int*)((char*)ws + codes_bytes(p.K, p.T));
        if (p.xt == XT_F32)
            x_code_kernel<XT_F32><<<p.T, 512, 0, s>>>(p.X, p.K, xq, xs);
        else if (p.xt == XT_F16)
            x_code_kernel<XT_F16><<<p.T, 512, 0, s>>>(p.X, p.K, xq, xs);
        else
            x_code_kernel<XT_BF16><<<p.T, 512, 0, s>>>(p.X, p.K, xq, xs);
    }
    if (fuse)
        p.N <= kFusedRows ? launch_rows<1, 1, 16, kFusedLds>(p, s) : launch_rows<1, 2, 8, kFusedLds>(p, s);
    else if (p.T <= 16)
        launch_few<1, 8>(p, s);
    else if (p.T <= 32)
        launch_few<2, 4>(p, s);
    else if (p.T <= 48)
        launch_few<3, 4>(p, s);
    else if (p.T <= 64)
        launch_few<4, 4>(p, s);
    else if (streams(p.N, p.T))
        p.T <= 96 ? launch_few<6, 4>(p, s) : launch_few<8, 4>(p, s);
    else if (large_tiles(p.N, p.T))
        launch_tile<2, 4, 4, 2, 2>(p, s);
    else if (tiles_of(p.N, p.T, 128) > 256)
        launch_tile<2, 2, 2, 2, 2>(p, s);
    else if (tiles_of(p.N, p.T, 128) > 160)
        launch_tile<2, 2, 2, 2, 4>(p, s);
    else
        launch_tile<1, 2, 2, 1, 4>(p, s);
    if (p.splits > 1) w8a8_join_kernel<<<dim3((p.N + 255) / 256, p.T), 256, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace qg
