// experts.hip -- the experts' matrix products between dispatch and combine: grouped by expert over
// the ragged expert-major rows, bf16 or e4m3 with block scales, plain or with the SwiGLU epilogue.
//
//   product   v[q][c] = sum_k a[q][k] w[e][c][k]                       bf16 operands, fp32 sums
//             v[q][c] = sum_b as[q][b] ws[e][c/128][b] p_b[q][c]       e4m3: p_b the fp32 sum over the
//                                                                      128 values k of block b
//   gated     h = g / (1 + exp(-g)) * u,  g = v[q][c], u = v[q][I + c]
#include "common.hpp"

namespace moe {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(8))) int i32x8;

// One product's operands, passed by value.  Rows of `a` and `w` are KB bytes; C is the number of
// output columns (the intermediate size I for the gated product, whose w has 2I rows).
struct Product {
    const uint8_t* a;
    const float* as;
    const uint8_t* w;
    const float* ws;
    const int32_t* off;
    uint8_t* out;
    float* out_scale;
    int32_t* status;
    long B;       // rows per rank
    int KB, KS;   // bytes of a row; scales of a row (e4m3)
    int C;
    int L, rb, rc;
};

constexpr int kStepBytes = 128;   // of every row, per step over K: 64 bf16 or 128 e4m3 values
constexpr int kMaxExperts = 1024; // of all ranks
constexpr int kThreads = 256;

// A chunk of zeros: what lanes past the end of a row load in its last step.
__device__ __attribute__((aligned(16))) const uint8_t kZeros[16] = {0};

__device__ __forceinline__ void load_lds16(const uint8_t* src, uint8_t* dst) {
    __builtin_amdgcn_global_load_lds((const void*)src, (lds_void*)dst, 16, 0, 0);
}
__device__ __forceinline__ void load_lds4(const float* src, float* dst) {
    __builtin_amdgcn_global_load_lds((const void*)src, (lds_void*)dst, 4, 0, 0);
}

// Rows of expert x of the call (x counts over its ranks' local experts): the first row within the
// rank, and how many.  Offsets that are no offsets of B rows flag MOE_EINVAL and own no rows.
__device__ __forceinline__ int expert_rows(const Product& P, int x, int* first) {
    const int d = P.rb + x / P.L, l = x % P.L;
    const int32_t* o = P.off + (long)d * (P.L + 1) + l;
    const int lo = o[0], hi = o[1];
    *first = lo;
    if (lo < 0 || hi < lo || (long)hi > P.B) {
        set_status(P.status, MOE_EINVAL);
        return 0;
    }
    return hi - lo;
}

// fp32 -> e4m3, to nearest even, clamped to +-448; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3_code(float v) {
    const uint32_t sign = (__float_as_uint(v) >> 24) & 0x80u;
    if (v != v) return sign | 0x7Fu;
    const float a = fminf(fabsf(v), 448.0f);
    if (a < 0.015625f) return sign | (uint32_t)__builtin_rintf(a * 512.0f);
    uint32_t b = __float_as_uint(a);
    b += 0x7FFFFu + ((b >> 20) & 1u);
    return sign | ((b >> 20) - (120u << 3));
}

__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// A block computes tiles of BM = 16 MT rows x BN = 16 NT WN weight rows with WN waves side by side
// along the weight rows.  The matrix instruction takes the weights as its first operand, so that a
// lane holds four neighbouring output columns of one row, and its row's scale is one number.  For
// the gated product the tile's weight rows alternate, 16 gate rows and 16 up rows, so that both
// factors of a column meet in the same register index of the same lane.
template <bool FP8, bool GATED, int MT, int NT, int WN>
__global__ __launch_bounds__(64 * WN) void k_experts(Product P) {
    constexpr int BM = 16 * MT, BN = 16 * NT * WN, T = 64 * WN;
    constexpr int kCols = GATED ? BN / 2 : BN;  // output columns of a tile
    __shared__ __attribute__((aligned(16))) uint8_t tile[(BM + BN) * kStepBytes];
    __shared__ float scl[T];
    __shared__ int base[kMaxExperts + 1];
    __shared__ float amax_of[WN][BM];
    const int lane = lane_id(), wave = wave_id();
    const int X = P.rc * P.L;
    const int ntn = (P.C + kCols - 1) / kCols;
    // tiles before each expert's
    for (int x = threadIdx.x; x < X; x += T) {
        int first;
        base[x] = (expert_rows(P, x, &first) + BM - 1) / BM;
    }
    __syncthreads();
    if (wave == 0) wave_excl_scan_array(base, base, X);
    __syncthreads();
    const long tiles = (long)base[X] * ntn;
    for (long t = blockIdx.x; t < tiles; t += gridDim.x) {
        // the expert whose tiles hold t: the last with base[x] * ntn <= t
        int x = 0;
        for (int s = 512; s > 0; s >>= 1)
            if (x + s < X && (long)base[x + s] * ntn <= t) x += s;
        const long in = t - (long)base[x] * ntn;
        const int mts = base[x + 1] - base[x];
        const int n0 = (int)(in / mts) * kCols, m0 = (int)(in % mts) * BM;
        int first;
        const int cnt = expert_rows(P, x, &first);
        const int d = P.rb + x / P.L;
        const long e = (long)d * P.L + x % P.L;
        const long row0 = (long)d * P.B + first;
        const int wrows = GATED ? 2 * P.C : P.C;
        const uint8_t* w = P.w + e * wrows * P.KB;

        f32x4 acc[NT][MT];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

        const int steps = (P.KB + kStepBytes - 1) / kStepBytes;
        for (int k = 0; k < steps; ++k) {
            // lane l of an instruction that fills rows 8i .. 8i+7 lands at row l/8, place l%8; it
            // fetches the row's 16-byte chunk (l%8) ^ (l/8), so that the reads below spread over the
            // LDS banks
            const int chunk = (lane & 7) ^ (lane >> 3);
            const int kb = k * kStepBytes + chunk * 16;
            for (int i = wave; i < (BM + BN) / 8; i += WN) {
                const int r = i * 8 + (lane >> 3);
                const uint8_t* src;
                if (r < BM) {
                    const int m = m0 + r < cnt ? m0 + r : cnt - 1;
                    src = P.a + (row0 + m) * P.KB + kb;
                } else {
                    const int q = r - BM;
                    int c = GATED ? n0 + (q >> 5) * 16 + (q & 15) : n0 + q;
                    c = c < P.C ? c : P.C - 1;
                    src = w + (long)(GATED && (q & 16) ? P.C + c : c) * P.KB + kb;
                }
                load_lds16(kb < P.KB ? src : kZeros, tile + i * 1024);
            }
            if constexpr (FP8) {
                // the rows' scales of this step, then the tile's weight blocks'
                const int i = threadIdx.x;
                const int m = m0 + i < cnt ? m0 + i : cnt - 1;
                const float* src = P.as + (row0 + m) * P.KS + k;
                if (i >= BM) {
                    const int j = i - BM, blocks = (wrows + 127) / 128;
                    int b = GATED ? (n0 + (j & 1) * P.C) / 128 : n0 / 128 + j;
                    b = b < blocks ? b : blocks - 1;
                    src = P.ws + (e * blocks + b) * P.KS + k;
                }
                load_lds4(src, scl + wave * 64);
            }
            __syncthreads();
            const int r16 = lane & 15, g = lane >> 4;
            float sr[MT], sw[2];
            if constexpr (FP8) {
#pragma unroll
                for (int j = 0; j < MT; ++j) sr[j] = scl[j * 16 + r16];
                sw[0] = scl[BM + (GATED ? 0 : wave * NT * 16 / 128)];
                sw[1] = GATED ? scl[BM + 1] : sw[0];
            }
            // row r's chunk c lies at place c ^ (r % 8); a lane takes chunks g and g + 4 of its row
            const int p0 = (g ^ (r16 & 7)) * 16, p1 = ((g + 4) ^ (r16 & 7)) * 16;
            i32x4 b[MT][2];
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                const uint8_t* row = tile + (j * 16 + r16) * kStepBytes;
                b[j][0] = *(const i32x4*)(row + p0);
                b[j][1] = *(const i32x4*)(row + p1);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const uint8_t* row = tile + (BM + (wave * NT + i) * 16 + r16) * kStepBytes;
                const i32x4 a0 = *(const i32x4*)(row + p0), a1 = *(const i32x4*)(row + p1);
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    if constexpr (FP8) {
                        const i32x8 A = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
                        const i32x8 Bv = __builtin_shufflevector(b[j][0], b[j][1], 0, 1, 2, 3, 4, 5, 6, 7);
                        const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            A, Bv, f32x4{0, 0, 0, 0}, 0, 0, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
                        const float s = sr[j] * sw[GATED ? (i & 1) : 0];
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(p[v], s, acc[i][j][v]);
                    } else {
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, a0), __builtin_bit_cast(bf16x8, b[j][0]), acc[i][j], 0, 0, 0);
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, a1), __builtin_bit_cast(bf16x8, b[j][1]), acc[i][j], 0, 0, 0);
                    }
                }
            }
            __syncthreads();
        }
        // epilogue: the lane's row of each 16-row group, four columns of each 16-column group
        const int r16 = lane & 15, c4 = (lane >> 4) * 4;
        if constexpr (!GATED) {
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                const int m = m0 + j * 16 + r16;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int c = n0 + (wave * NT + i) * 16 + c4;
                    if (m >= cnt || c >= P.C) continue;
                    uint2 v;
                    v.x = f32_to_bf16(acc[i][j][0]) | f32_to_bf16(acc[i][j][1]) << 16;
                    v.y = f32_to_bf16(acc[i][j][2]) | f32_to_bf16(acc[i][j][3]) << 16;
                    *(uint2*)(P.out + ((row0 + m) * P.C + c) * 2) = v;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int i = 0; i < NT; i += 2)
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[i][j][v] = swiglu(acc[i][j][v], acc[i + 1][j][v]);
            if constexpr (FP8) {
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    float m = 0.0f;
#pragma unroll
                    for (int i = 0; i < NT; i += 2)
#pragma unroll
                        for (int v = 0; v < 4; ++v) m = fmaxf(m, fabsf(acc[i][j][v]));
                    m = fmaxf(m, __shfl_xor(m, 16, kWave));
                    m = fmaxf(m, __shfl_xor(m, 32, kWave));
                    if (lane < 16) amax_of[wave][j * 16 + lane] = m;
                }
                __syncthreads();
            }
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                const int m = m0 + j * 16 + r16;
                float sc = 1.0f;
                if constexpr (FP8) {
                    float a = 0.0f;
#pragma unroll
                    for (int q = 0; q < WN; ++q) a = fmaxf(a, amax_of[q][j * 16 + r16]);
                    sc = a > 0.0f ? a / 448.0f : 1.0f;
                    if (wave == 0 && lane < 16 && m < cnt)
                        P.out_scale[(row0 + m) * (P.C / 128) + n0 / 128] = sc;
                }
#pragma unroll
                for (int i = 0; i < NT; i += 2) {
                    const int c = n0 + (wave * NT + i) * 8 + c4;
                    if (m >= cnt || c >= P.C) continue;
                    const f32x4 h = acc[i][j];
                    if constexpr (FP8) {
                        *(uint32_t*)(P.out + (row0 + m) * P.C + c) =
                            e4m3_code(h[0] / sc) | e4m3_code(h[1] / sc) << 8 | e4m3_code(h[2] / sc) << 16 |
                            e4m3_code(h[3] / sc) << 24;
                    } else {
                        uint2 v;
                        v.x = f32_to_bf16(h[0]) | f32_to_bf16(h[1]) << 16;
                        v.y = f32_to_bf16(h[2]) | f32_to_bf16(h[3]) << 16;
                        *(uint2*)(P.out + ((row0 + m) * P.C + c) * 2) = v;
                    }
                }
            }
            if constexpr (FP8) __syncthreads();
        }
    }
}

// ------------------------------------------------------------------ launchers

// gated: columns C of a w with 2C rows; out holds bf16 rows, or for a gated e4m3 product codes and
// out_scale.
hipError_t launch_experts(const Dims& D, bool gated, int K, int C, const void* a, const float* as, const void* w,
                          const float* ws, const int32_t* off, void* out, float* out_scale, hipStream_t st) {
    Product P;
    P.a = (const uint8_t*)a;
    P.as = as;
    P.w = (const uint8_t*)w;
    P.ws = ws;
    P.off = off;
    P.out = (uint8_t*)out;
    P.out_scale = out_scale;
    P.status = D.status;
    P.B = D.B;
    P.KB = D.fp8 ? K : 2 * K;
    P.KS = K / 128;
    P.C = C;
    P.L = D.L;
    P.rb = D.rb;
    P.rc = D.rc;
    constexpr int MT = 4, NT = 4, WN = 4;
    const long mts = (recv_rows_bound(D) + 16 * MT - 1) / (16 * MT) + (long)D.rc * D.L;
    const int cols = gated ? 8 * NT * WN : 16 * NT * WN;
    const long tiles = mts * ((C + cols - 1) / cols);
    const dim3 grid((unsigned)(tiles < 1024 ? tiles : 1024)), block(64 * WN);
    if (D.fp8 && gated) hipLaunchKernelGGL((k_experts<true, true, MT, NT, WN>), grid, block, 0, st, P);
    else if (D.fp8) hipLaunchKernelGGL((k_experts<true, false, MT, NT, WN>), grid, block, 0, st, P);
    else if (gated) hipLaunchKernelGGL((k_experts<false, true, MT, NT, WN>), grid, block, 0, st, P);
    else hipLaunchKernelGGL((k_experts<false, false, MT, NT, WN>), grid, block, 0, st, P);
    return hipGetLastError();
}

}  // namespace moe
