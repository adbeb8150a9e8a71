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

constexpr int kStepBytes = 128;    // of every row, per step over K: 64 bf16 or 128 e4m3 values
constexpr int kMaxExperts = 1024;  // of all ranks
constexpr int kCUs = 256;
constexpr int kWaves = 8;
constexpr int kThreads = kWaves * kWave;
constexpr int kRingBytes = 150 << 10;
constexpr int kEpiBytes = 4 << 10;
constexpr int kGroupTiles = 8;     // row tiles that share a weight tile before the next one

// A chunk of zeros: what lanes past the end of a row load in its last step.
__device__ __attribute__((aligned(16))) const uint8_t kZeros[16] = {0};

// The shape of a tile: BM rows x BN weight rows by WM x WN x KP waves (KP: waves that share a
// tile's part and take every KP-th step), through a ring of S stages of KP steps each.
template <int BM_, int BN_, int WM_, int WN_, int KP_, int S_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, KP = KP_, S = S_;
    static_assert(WM * WN * KP == kWaves, "eight waves");
    static constexpr int MT = BM / 16 / WM, NT = BN / 16 / WN;  // 16 x 16 parts of a wave
    static constexpr int kFillsPerStep = (BM + BN) / 8;         // loads of 8 rows
    static constexpr int kFills = KP * kFillsPerStep;
    static constexpr int kPerWave = (kFills + kWaves - 1) / kWaves;
    static constexpr int kTileBytes = KP * (BM + BN) * kStepBytes;
    // the scales of a stage (e4m3): a row of kThreads floats; KP steps of BM + 2 of them are used
    template <bool FP8>
    static constexpr int stage() { return kTileBytes + (FP8 ? kThreads * 4 : 0); }
    static_assert(KP * (BM + 2) <= kThreads, "a stage's scales");
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A barrier that waits for the wave's LDS accesses but not for its loads and stores in flight.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Waits until at most N of the wave's loads and stores are in flight (loads end in order).  Not the
// builtin: after __builtin_amdgcn_s_waitcnt(vmcnt(0)) the compiler made the LDS reads of the
// two-stage ring wait for the loads issued since, which the other stage receives.
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "six bits");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
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

// What tile t is of: its expert's rows and matrix, and where in them it lies.
struct Place {
    int cnt, m0, n0;
    int end;    // of the tile's rows
    long row0;  // the expert's first row in the row arrays
    long e;
};

template <class T, bool GATED>
__device__ __forceinline__ Place place_of(const Product& P, const int* base, int X, int ntn, int t) {
    // the last expert with base[x] <= q: 16 at a time, then one by one
    const int q = t / ntn, lane = lane_id();
    int i = lane * 16;
    const int c = __popcll(ballot(i < X && base[i < X ? i : 0] <= q)) - 1;
    i = c * 16 + lane;
    const int x = c * 16 + __popcll(ballot(lane < 16 && i < X && base[i < X ? i : 0] <= q)) - 1;
    const int b0 = uniform(base[x]), mts = uniform(base[x + 1]) - b0;
    // row tiles in groups: within a group every row tile meets a weight tile before the next one
    // comes, so that both stay in the XCD's cache while its CUs use them
    const int in = t - b0 * ntn, g = in / (kGroupTiles * ntn), r = in - g * kGroupTiles * ntn;
    const int left = mts - g * kGroupTiles, gm = left < kGroupTiles ? left : kGroupTiles;
    Place p;
    int first;
    p.cnt = uniform(expert_rows(P, x, &first));
    // the expert's tiles share its rows evenly, in parts of 16
    const int rows = ((p.cnt + mts - 1) / mts + 15) & ~15;
    p.m0 = (g * kGroupTiles + r % gm) * rows;
    p.n0 = r / gm * (GATED ? T::BN / 2 : T::BN);
    p.end = p.m0 + rows < p.cnt ? p.m0 + rows : p.cnt;
    const int d = P.rb + x / P.L;
    p.e = (long)d * P.L + x % P.L;
    p.row0 = (long)d * P.B + uniform(first);
    return p;
}

// Where a wave loads a stage of a tile from: the tile's first row, weight row and (gated) up row, an
// offset of the lane for each fill, and the lane's scale.
template <class T>
struct Source {
    const uint8_t *rows, *weights, *ups;
    uint32_t off[T::kPerWave];
    const float* scale;
};

// Fill i = wave + 8 j of a stage brings rows 8 (i % kFillsPerStep) .. + 7 of step i / kFillsPerStep.
template <class T>
struct Fill {
    int kp, r;  // step; first of its rows: BM rows, then BN weight rows
    __device__ __forceinline__ Fill(int wave, int j) {
        const int i = (wave & 7) + j * kWaves;
        kp = T::KP == 1 ? 0 : i / T::kFillsPerStep;
        r = (i - kp * T::kFillsPerStep) * 8;
    }
    template <bool GATED>
    __device__ __forceinline__ const uint8_t* of(const uint8_t* rows, const uint8_t* weights, const uint8_t* ups) const {
        return r < T::BM ? rows : GATED && (r - T::BM & 16) ? ups : weights;
    }
};

__device__ __forceinline__ void load_lds16(const uint8_t* src, uint8_t* dst) {
    __builtin_amdgcn_global_load_lds((const void*)src, (lds_void*)dst, 16, 0, 0);
}
__device__ __forceinline__ void load_lds4(const float* src, float* dst) {
    __builtin_amdgcn_global_load_lds((const void*)src, (lds_void*)dst, 4, 0, 0);
}

// Lane l of a fill lands at row l / 8, place l % 8, and fetches the row's 16-byte chunk (l % 8) ^ (l / 8):
// the reads of a 16-row part then spread over the LDS banks.  Rows past an expert's last repeat it;
// weight rows past the last repeat it too.  For the gated product the weight rows of a tile alternate,
// 16 gate rows and 16 up rows.
template <bool FP8, bool GATED, class T>
__device__ __forceinline__ void aim(const Product& P, const Place& p, Source<T>& s) {
    const int lane = lane_id(), wave = uniform(wave_id());
    const int wrows = GATED ? 2 * P.C : P.C;
    const int chunk = (lane & 7) ^ (lane >> 3), r8 = lane >> 3;
    s.rows = P.a + (p.row0 + p.m0) * P.KB;
    s.weights = P.w + (p.e * wrows + p.n0) * P.KB;
    s.ups = s.weights + (long)P.C * P.KB;
#pragma unroll
    for (int j = 0; j < T::kPerWave; ++j) {
        const Fill<T> f(wave, j);
        const int q = f.r - T::BM;
        const bool tok = q < 0;
        const int r = (tok ? f.r : GATED ? (q >> 5) * 16 + (q & 15) : q) + r8;
        const int last = tok ? p.cnt - 1 - p.m0 : P.C - 1 - p.n0;
        s.off[j] = (uint32_t)(r < last ? r : last) * P.KB + f.kp * kStepBytes + chunk * 16;
    }
    if constexpr (FP8) {
        const int i = threadIdx.x, kp = i / (T::BM + 2), r = i - kp * (T::BM + 2);
        const int blocks = (wrows + 127) / 128;
        if (r < T::BM || kp >= T::KP) {
            const int m = p.m0 + r < p.cnt ? p.m0 + r : p.cnt - 1;
            s.scale = P.as + (p.row0 + m) * P.KS + (kp < T::KP ? kp : 0);
        } else {
            int b = GATED ? (p.n0 + (r - T::BM) * P.C) / 128 : p.n0 / 128 + (r - T::BM);
            b = b < blocks ? b : blocks - 1;
            s.scale = P.ws + (p.e * blocks + b) * P.KS + kp;
        }
    }
}

// Loads stage k of the tile that `src` aims at into `wr`.
template <bool FP8, bool GATED, class T>
__device__ __forceinline__ void fetch_stage(uint8_t* wr, const Product& P, const Source<T>& src, int k) {
    const int lane = lane_id(), wave = uniform(wave_id());
    const int kb = k * T::KP * kStepBytes;
    const uint8_t *rows = src.rows + kb, *weights = src.weights + kb, *ups = src.ups + kb;
    if ((FP8 && T::KP == 1) || kb + T::KP * kStepBytes <= P.KB) {
#pragma unroll
        for (int j = 0; j < T::kPerWave; ++j) {
            const Fill<T> f(wave, j);
            if (T::kFills % kWaves == 0 || wave + j * kWaves < T::kFills)
                load_lds16(f.template of<GATED>(rows, weights, ups) + src.off[j], wr + (wave + j * kWaves) * 1024);
        }
    } else {  // the last stage of a row: zeros from the row's end on
        const int chunk = (lane & 7) ^ (lane >> 3);
#pragma unroll
        for (int j = 0; j < T::kPerWave; ++j) {
            const Fill<T> f(wave, j);
            uint32_t off = src.off[j];
            asm volatile("" : "+v"(off));  // keeps this path's addresses out of the other's registers
            const bool in = kb + f.kp * kStepBytes + chunk * 16 < P.KB;
            if (T::kFills % kWaves == 0 || wave + j * kWaves < T::kFills)
                load_lds16(in ? f.template of<GATED>(rows, weights, ups) + off : kZeros, wr + (wave + j * kWaves) * 1024);
        }
    }
    if constexpr (FP8) {
        // a step past the last reads the row's last scale (its codes are zeros)
        const int kp = threadIdx.x / (T::BM + 2);
        const int ks = k * T::KP, over = ks + (kp < T::KP ? kp : 0) - (P.KS - 1);
        load_lds4(src.scale + ks - (over > 0 ? over : 0), (float*)(wr + T::kTileBytes) + wave * 64);
    }
}

// One stage: the loads of stage k of a tile into `wr` (if `fetch`), and the products of the stage in
// `rd`.  The two never overlap; saying so (__restrict__ on both) keeps the compiler from making the
// reads wait for the loads.
template <bool FP8, bool GATED, class T>
__device__ __forceinline__ void stage_step(const uint8_t* __restrict__ rd, uint8_t* __restrict__ wr, const Product& P,
                                           const Source<T>& src, int k, bool fetch, f32x4 (&acc)[T::NT][T::MT]) {
    constexpr int MT = T::MT, NT = T::NT;
    const int lane = lane_id(), wave = uniform(wave_id());
    if (fetch) fetch_stage<FP8, GATED, T>(wr, P, src, k);
    const int r16 = lane & 15, g = lane >> 4;
    const int wm = wave / T::WN % T::WM, wn = wave % T::WN, kp = wave / (T::WM * T::WN);
    float sr[MT], sw[2];
    if constexpr (FP8) {
        const float* scl = (const float*)(rd + T::kTileBytes) + kp * (T::BM + 2);
#pragma unroll
        for (int j = 0; j < MT; ++j) sr[j] = scl[(j * T::WM + wm) * 16 + r16];
        sw[0] = scl[T::BM + (GATED ? 0 : wn * NT * 16 / 128)];
        sw[1] = GATED ? scl[T::BM + 1] : sw[0];
    }
    // row r's chunk c lies at place c ^ (r % 8); a lane takes chunks g and g + 4 of its row
    const int p0 = (g ^ (r16 & 7)) * 16, p1 = p0 ^ 64;
    const uint8_t* ta = rd + (kp * (T::BM + T::BN) + wm * 16 + r16) * kStepBytes;
    constexpr int kNext = T::WM * 16 * kStepBytes;  // to the wave's next part
    const uint8_t* tw = rd + (kp * (T::BM + T::BN) + T::BM + wn * NT * 16 + r16) * kStepBytes;
    i32x4 w[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        w[i][0] = *(const i32x4*)(tw + i * 16 * kStepBytes + p0);
        w[i][1] = *(const i32x4*)(tw + i * 16 * kStepBytes + p1);
    }
    i32x4 b[2][2];
    b[0][0] = *(const i32x4*)(ta + p0);
    b[0][1] = *(const i32x4*)(ta + p1);
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        // the next part's rows are read while this one's products run; no further ahead, for the
        // registers' sake
        if (j + 1 < MT) {
            b[(j + 1) & 1][0] = *(const i32x4*)(ta + (j + 1) * kNext + p0);
            b[(j + 1) & 1][1] = *(const i32x4*)(ta + (j + 1) * kNext + p1);
        }
        const i32x4 b0 = b[j & 1][0], b1 = b[j & 1][1];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if constexpr (FP8) {
                const i32x8 A = __builtin_shufflevector(w[i][0], w[i][1], 0, 1, 2, 3, 4, 5, 6, 7);
                const i32x8 B = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
                const f32x4 p =
                    __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
                const float s = sr[j] * sw[GATED ? (i & 1) : 0];
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(p[v], s, acc[i][j][v]);
                // here, and not after all products: the partial sums would need registers of their own
                asm volatile("" : "+v"(acc[i][j]));
            } else {
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, w[i][0]), __builtin_bit_cast(bf16x8, b0), acc[i][j], 0, 0, 0);
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, w[i][1]), __builtin_bit_cast(bf16x8, b1), acc[i][j], 0, 0, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// A tile's results: the lane's row of each 16-row part, four neighbouring columns of each 16-column
// part.  `epi`: LDS apart from the ring.
template <bool FP8, bool GATED, class T>
__device__ __forceinline__ void write_tile(const Product& P, const Place& p, f32x4 (&acc)[T::NT][T::MT], float* epi) {
    constexpr int MT = T::MT, NT = T::NT;
    const int lane = lane_id(), wave = uniform(wave_id());
    const int wm = wave / T::WN % T::WM, wn = wave % T::WN, kp = wave / (T::WM * T::WN);
    const int r16 = lane & 15, c4 = (lane >> 4) * 4;
    if constexpr (T::KP > 1) {
        // the waves that took a part's steps in turn add up in their order, kAtOnce 16 x 16 parts at
        // a time: each of the others leaves its sums for the first
        constexpr int kAtOnce = kEpiBytes / (T::WM * T::WN * 16 * kWave);
        static_assert(kAtOnce >= 1, "room for the sums of a part");
        f32x4* mine = (f32x4*)epi + wave % (T::WM * T::WN) * kAtOnce * kWave + lane;
        for (int q = 1; q < T::KP; ++q) {
#pragma unroll
            for (int f = 0; f < NT * MT; f += kAtOnce) {
                if (kp == q) {
#pragma unroll
                    for (int u = f; u < f + kAtOnce && u < NT * MT; ++u) mine[(u - f) * kWave] = acc[u / MT][u % MT];
                }
                lds_barrier();
                if (kp == 0) {
#pragma unroll
                    for (int u = f; u < f + kAtOnce && u < NT * MT; ++u) acc[u / MT][u % MT] += mine[(u - f) * kWave];
                }
                lds_barrier();
            }
        }
    }
    const bool writes = kp == 0;
    if constexpr (!GATED) {
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int m = p.m0 + (j * T::WM + wm) * 16 + r16;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int c = p.n0 + (wn * NT + i) * 16 + c4;
                if (!writes || m >= p.end || c >= P.C) continue;
                uint2 v;
                v.x = f32_to_bf16(acc[i][j][0]) | f32_to_bf16(acc[i][j][1]) << 16;
                v.y = f32_to_bf16(acc[i][j][2]) | f32_to_bf16(acc[i][j][3]) << 16;
                *(uint2*)(P.out + ((p.row0 + m) * P.C + c) * 2) = v;
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
            static_assert(T::BN == 256 && T::KP == 1, "a tile holds a whole block of 128 columns");
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < NT; i += 2)
#pragma unroll
                    for (int v = 0; v < 4; ++v) m = fmaxf(m, fabsf(acc[i][j][v]));
                m = fmaxf(m, __shfl_xor(m, 16, kWave));
                m = fmaxf(m, __shfl_xor(m, 32, kWave));
                if (lane < 16) epi[wn * T::BM + (j * T::WM + wm) * 16 + lane] = m;
            }
            lds_barrier();
        }
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int m = p.m0 + (j * T::WM + wm) * 16 + r16;
            float sc = 1.0f;
            if constexpr (FP8) {
                float a = 0.0f;
#pragma unroll
                for (int q = 0; q < T::WN; ++q) a = fmaxf(a, epi[q * T::BM + (j * T::WM + wm) * 16 + r16]);
                sc = a > 0.0f ? a / 448.0f : 1.0f;
                if (wn == 0 && lane < 16 && m < p.end) P.out_scale[(p.row0 + m) * (P.C / 128) + p.n0 / 128] = sc;
            }
#pragma unroll
            for (int i = 0; i < NT; i += 2) {
                const int c = p.n0 + (wn * NT + i) * 8 + c4;
                if (!writes || m >= p.end || c >= P.C) continue;
                const f32x4 h = acc[i][j];
                if constexpr (FP8) {
                    *(uint32_t*)(P.out + (p.row0 + m) * P.C + c) = e4m3_code(h[0] / sc) | e4m3_code(h[1] / sc) << 8 |
                                                                   e4m3_code(h[2] / sc) << 16 |
                                                                   e4m3_code(h[3] / sc) << 24;
                } else {
                    uint2 v;
                    v.x = f32_to_bf16(h[0]) | f32_to_bf16(h[1]) << 16;
                    v.y = f32_to_bf16(h[2]) | f32_to_bf16(h[3]) << 16;
                    *(uint2*)(P.out + ((p.row0 + m) * P.C + c) * 2) = v;
                }
            }
        }
        if constexpr (FP8) lds_barrier();  // the next tile's maxima
    }
}

// The block's tiles, v, v + G, ..., as one run of stages: the loads run S - 1 stages ahead of the
// products, across the ends of tiles.
template <bool FP8, bool GATED, class T>
__device__ __forceinline__ void run_tiles(const Product& P, uint8_t* ring, const int* base, float* epi, int X, int v,
                                          int G) {
    constexpr int kStage = T::template stage<FP8>(), S = T::S;
    static_assert(S * kStage <= kRingBytes, "the ring");
    constexpr int kLoads = T::kPerWave + (FP8 ? 1 : 0);  // of a stage, at most
    // waves with fewer fills than others wait for one stage more than they need
    constexpr int kFew = T::kFills / kWaves + (FP8 ? 1 : 0);
    const int ntn = (P.C + (GATED ? T::BN / 2 : T::BN) - 1) / (GATED ? T::BN / 2 : T::BN);
    const int tiles = base[X] * ntn;
    if (v >= tiles) return;
    const int stages = (P.KB + T::KP * kStepBytes - 1) / (T::KP * kStepBytes);
    const long total = (long)((tiles - 1 - v) / G + 1) * stages;
    const bool many = uniform(wave_id()) < T::kFills % kWaves;
    f32x4 acc[T::NT][T::MT];
    Source<T> src;
    Place p = place_of<T, GATED>(P, base, X, ntn, v);
    aim<FP8, GATED, T>(P, p, src);
    int lt = v, lk = 0, ct = v, ck = 0;  // tile and stage of the loads and of the products
    int rslot = 0, wslot = 0;
    auto zero = [&] {
#pragma unroll
        for (int i = 0; i < T::NT; ++i)
#pragma unroll
            for (int j = 0; j < T::MT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    };
    zero();
    auto advance = [&] {
        ++lk;
        wslot = wslot == S - 1 ? 0 : wslot + 1;
        if (lk == stages) {
            lk = 0;
            lt += G;
            if (lt < tiles) aim<FP8, GATED, T>(P, place_of<T, GATED>(P, base, X, ntn, lt), src);
        }
    };
    for (int n = 0; n < S - 1 && n < total; ++n) {
        fetch_stage<FP8, GATED, T>(ring + wslot * kStage, P, src, lk);
        advance();
    }
    for (long n = 0; n < total; ++n) {
        if (n + S - 1 <= total) {
            if (T::kFills % kWaves && many) wait_loads<(S - 2) * kLoads>();
            else wait_loads<(S - 2) * (T::kFills % kWaves ? kFew : kLoads)>();
        } else {
            wait_loads<0>();
        }
        lds_barrier();
        const bool fetch = n + S - 1 < total;
        stage_step<FP8, GATED, T>(ring + rslot * kStage, ring + wslot * kStage, P, src, lk, fetch, acc);
        rslot = rslot == S - 1 ? 0 : rslot + 1;
        if (fetch) advance();
        if (++ck == stages) {
            write_tile<FP8, GATED, T>(P, p, acc, epi);
            zero();
            ck = 0;
            ct += G;
            if (ct < tiles) p = place_of<T, GATED>(P, base, X, ntn, ct);
        }
    }
    lds_barrier();
}

// The tiles, from few rows and columns to many.  The gated product needs two 16-row parts of a tile's
// weight rows in each wave (gate and up), and with e4m3 operands 256 of them in a tile: it quantises
// blocks of 128 output columns.
constexpr int kTiles = 11, kLevels = 5;
enum { kPlain, kGated, kWide };
template <int KIND, int I> struct TileOf;
template <> struct TileOf<kPlain, 0> { typedef Tile<16, 32, 1, 2, 4, 5> type; };
template <> struct TileOf<kPlain, 1> { typedef Tile<32, 32, 2, 2, 2, 8> type; };
template <> struct TileOf<kPlain, 2> { typedef Tile<16, 64, 1, 4, 2, 6> type; };
template <> struct TileOf<kPlain, 3> { typedef Tile<64, 64, 2, 4, 1, 8> type; };
template <> struct TileOf<kPlain, 4> { typedef Tile<16, 128, 1, 8, 1, 7> type; };
template <> struct TileOf<kPlain, 5> { typedef Tile<32, 128, 1, 8, 1, 6> type; };
template <> struct TileOf<kPlain, 6> { typedef Tile<64, 128, 2, 4, 1, 5> type; };
template <> struct TileOf<kGated, 0> { typedef Tile<16, 32, 1, 1, 8, 3> type; };
template <> struct TileOf<kGated, 1> { typedef Tile<32, 32, 2, 1, 4, 4> type; };
template <> struct TileOf<kGated, 2> { typedef Tile<16, 64, 1, 2, 4, 3> type; };
template <> struct TileOf<kGated, 3> { typedef Tile<64, 64, 4, 2, 1, 8> type; };
template <> struct TileOf<kGated, 4> { typedef Tile<16, 128, 1, 4, 2, 4> type; };
template <> struct TileOf<kGated, 5> { typedef Tile<32, 128, 2, 4, 1, 7> type; };
template <> struct TileOf<kGated, 6> { typedef Tile<64, 128, 2, 4, 1, 6> type; };
template <> struct TileOf<kWide, 4> { typedef Tile<16, 256, 1, 8, 1, 4> type; };
template <> struct TileOf<kWide, 5> { typedef Tile<32, 256, 1, 8, 1, 3> type; };
template <> struct TileOf<kWide, 6> { typedef Tile<64, 256, 1, 8, 1, 3> type; };
template <> struct TileOf<kWide, 7> { typedef Tile<128, 256, 2, 4, 1, 3> type; };
template <int KIND> struct TileOf<KIND, 7> { typedef Tile<128, 128, 2, 4, 1, 4> type; };
template <int KIND> struct TileOf<KIND, 8> { typedef Tile<160, 256, 2, 4, 1, 2> type; };
template <int KIND> struct TileOf<KIND, 9> { typedef Tile<192, 256, 2, 4, 1, 2> type; };
template <int KIND> struct TileOf<KIND, 10> { typedef Tile<256, 256, 2, 4, 1, 2> type; };

// At each level an expert's rows make as few row tiles as fit `most` rows each (0: the largest tile;
// further levels smaller ones, for products that would leave CUs without a tile), and the tiles take
// the least height that holds their even share.
template <bool WIDE>
__device__ __forceinline__ int level_rows(int level) {
    return level == 0 ? 256 : level == 1 ? 128 : WIDE || level <= 3 ? 64 : 32;
}
template <bool WIDE>
__device__ __forceinline__ int row_tiles(int rows, int level) {
    return (rows + level_rows<WIDE>(level) - 1) / level_rows<WIDE>(level);
}
template <bool WIDE>
__device__ __forceinline__ int tile_of(int rows, int level) {
    const int mts = row_tiles<WIDE>(rows, level), n = (rows + mts - 1) / (mts > 0 ? mts : 1);
    if (!WIDE && level == 4) return n > 16 ? 1 : 0;
    if (!WIDE && level == 3) return n > 16 ? 3 : 2;
    return n > 192 ? 10 : n > 160 ? 9 : n > 128 ? 8 : n > 64 ? 7 : n > 32 ? 6 : n > 16 ? 5 : 4;
}

// Columns of weight rows of a tile, and the time of a step over K, in cycles.
template <bool WIDE>
__device__ __forceinline__ int tile_width(int i) {
    return WIDE || i >= 8 ? 256 : i >= 4 ? 128 : i >= 2 ? 64 : 32;
}
template <bool WIDE>
__device__ __forceinline__ int tile_time(int i, int rows) {
    if (i >= 8) return 1000 + 8 * rows;
    if (WIDE) return 700 + 8 * rows;
    return i >= 4 ? 450 + 4 * rows : i >= 2 ? 300 + 2 * rows : 200 + rows;
}

// base[x] = row tiles of tile i of the experts before x.
template <bool WIDE>
__device__ __forceinline__ void scan_tiles(const int* rows, int level, int tile, int X, int* base, int* part) {
    lds_barrier();  // the last tile's run is done with base
    int n[2], v = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int x = 2 * threadIdx.x + i;
        n[i] = rows[i] > 0 && tile_of<WIDE>(rows[i], level) == tile ? row_tiles<WIDE>(rows[i], level) : 0;
        v += n[i];
    }
    const int inc = wave_incl_scan(v);
    if (lane_id() == kWave - 1) part[wave_id()] = inc;
    lds_barrier();
    int before = inc - v;
    for (int w = 0; w < wave_id(); ++w) before += part[w];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int x = 2 * threadIdx.x + i;
        if (x <= X) base[x] = before;
        before += n[i];
    }
    if (threadIdx.x == kThreads - 1) base[kMaxExperts] = before;
    lds_barrier();
}

template <bool FP8, bool GATED>
__global__ __launch_bounds__(kThreads) void k_experts(Product P) {
    constexpr bool WIDE = FP8 && GATED;
    constexpr int KIND = WIDE ? kWide : GATED ? kGated : kPlain;
    __shared__ __attribute__((aligned(16))) uint8_t ring[kRingBytes];
    __shared__ __attribute__((aligned(16))) float epi[kEpiBytes / 4];
    __shared__ int base[kMaxExperts + 1];
    __shared__ int part[kWaves];
    __shared__ unsigned long long sum[kLevels];
    __shared__ int most[kLevels];
    __shared__ int present;
    const int X = P.rc * P.L, G = gridDim.x;
    // blocks of one XCD (the hardware deals blocks to the eight in turn) take neighbouring tiles
    const int per = G / 8, b = blockIdx.x;
    const int v = b < per * 8 ? b % 8 * per + b / 8 : b;
    if (threadIdx.x < kLevels) {
        sum[threadIdx.x] = 0;
        most[threadIdx.x] = 0;
    }
    if (threadIdx.x == 0) present = 0;
    lds_barrier();
    int rows[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int x = 2 * threadIdx.x + i;
        int first;
        if (x < X) rows[i] = expert_rows(P, x, &first);
    }
    // the level whose tiles end first: their times over all blocks, or the longest of them
    constexpr int levels = WIDE ? 3 : kLevels;
    for (int l = 0; l < levels; ++l) {
        long t = 0;
        int longest = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (rows[i] == 0) continue;
            const int tile = tile_of<WIDE>(rows[i], l), mts = row_tiles<WIDE>(rows[i], l);
            const int cols = GATED ? tile_width<WIDE>(tile) / 2 : tile_width<WIDE>(tile);
            const int one = tile_time<WIDE>(tile, (rows[i] + mts - 1) / mts);
            t += (long)mts * ((P.C + cols - 1) / cols) * one;
            longest = one > longest ? one : longest;
        }
        if (longest) {
            atomicAdd(&sum[l], (unsigned long long)t);
            atomicMax(&most[l], longest);
        }
    }
    lds_barrier();
    int level = 0;
    long least = 0;
    for (int l = 0; l < levels; ++l) {
        const long all = (long)sum[l] / G, t = all > most[l] ? all : most[l];
        if (l == 0 || t < least) {
            level = l;
            least = t;
        }
    }
    level = uniform(level);
#ifdef MOE_EXPERT_LEVEL
    level = MOE_EXPERT_LEVEL;
#endif
    int bits = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (rows[i] > 0) bits |= 1 << tile_of<WIDE>(rows[i], level);
    if (bits) atomicOr(&present, bits);
    lds_barrier();
    const int all = uniform(present);
    int done = 0;  // tiles so far: the next kind of tile begins at the block after them
    auto run = [&](auto tile, int i) {
        typedef decltype(tile) T;
        if (!(all >> i & 1)) return;
        scan_tiles<WIDE>(rows, level, i, X, base, part);
        int w = v - done % G;
        w = w < 0 ? w + G : w;
        run_tiles<FP8, GATED, T>(P, ring, base, epi, X, w, G);
        const int cols = GATED ? T::BN / 2 : T::BN;
        done += uniform(base[X]) * ((P.C + cols - 1) / cols);
    };
    run(typename TileOf<KIND, 10>::type(), 10);
    run(typename TileOf<KIND, 9>::type(), 9);
    run(typename TileOf<KIND, 8>::type(), 8);
    run(typename TileOf<KIND, 7>::type(), 7);
    run(typename TileOf<KIND, 6>::type(), 6);
    run(typename TileOf<KIND, 5>::type(), 5);
    run(typename TileOf<KIND, 4>::type(), 4);
    if constexpr (!WIDE) {
        run(typename TileOf<KIND, 3>::type(), 3);
        run(typename TileOf<KIND, 2>::type(), 2);
        run(typename TileOf<KIND, 1>::type(), 1);
        run(typename TileOf<KIND, 0>::type(), 0);
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
    // one block a CU (each takes nearly all of its LDS); fewer if there cannot be as many tiles
    const long mts = (recv_rows_bound(D) + 15) / 16 + (long)D.rc * D.L;
    const int cols = D.fp8 && gated ? 128 : gated ? 16 : 32;
    const long tiles = mts * ((C + cols - 1) / cols);
    const dim3 grid((unsigned)(tiles < kCUs ? tiles : kCUs)), block(kThreads);
    if (D.fp8 && gated) hipLaunchKernelGGL((k_experts<true, true>), grid, block, 0, st, P);
    else if (D.fp8) hipLaunchKernelGGL((k_experts<true, false>), grid, block, 0, st, P);
    else if (gated) hipLaunchKernelGGL((k_experts<false, true>), grid, block, 0, st, P);
    else hipLaunchKernelGGL((k_experts<false, false>), grid, block, 0, st, P);
    return hipGetLastError();
}

}  // namespace moe
