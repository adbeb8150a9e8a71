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
constexpr int kRingBytes = 147200;
constexpr int kEpiBytes = 4 << 10;
constexpr int kGroupTiles = 8;     // row tiles that share a weight tile before the next one

// A chunk of zeros: what lanes past the end of a row load in its last step.
__device__ __attribute__((aligned(16))) const uint8_t kZeros[16] = {0};

// The shape of a tile: BM rows x BN weight rows by WM x WN x KP waves (KP: waves that share a
// tile's part and take every KP-th step).  A stage is KP steps.  The rows go through a ring of SR
// stages, loaded by the first waves, the weights through one of SW, loaded by the last four: a wave
// waits for its loads in their order, so rows (short way, from the cache) and weights (long way, from
// memory) wait apart.  EARLY: a stage's weights are read into registers at its begin and their place
// refilled at once, not after the stage.
template <int BM_, int BN_, int WM_, int WN_, int KP_, int SR_, int SW_, bool EARLY_ = false>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, KP = KP_, SR = SR_, SW = SW_;
    static constexpr bool EARLY = EARLY_;
    static_assert(WM * WN * KP == kWaves, "eight waves");
    static constexpr int MT = BM / 16 / WM, NT = BN / 16 / WN;  // 16 x 16 parts of a wave
    // waves that load rows and weights, and the loads of 8 rows of each, a stage
    static constexpr int kRowFills = KP * BM / 8, kWeightFills = KP * BN / 8;
    static constexpr int WR = kRowFills < 4 ? kRowFills : 4, WW = 4;
    static constexpr int FR = kRowFills / WR, FW = kWeightFills / WW, F = FR > FW ? FR : FW;
    static_assert(FR * WR == kRowFills && FW * WW == kWeightFills, "whole fills");
    // stages that the loads run ahead
    static constexpr int kRowLead = SR - 1, kWeightLead = EARLY ? SW : SW - 1;
    static constexpr int kRowSlot = KP * BM * kStepBytes, kWeightSlot = KP * BN * kStepBytes;
    // e4m3: the scales of four steps, 16 bytes for each row and for the tile's two weight blocks
    static constexpr int kScaleLoads = (BM + 2 + kWave - 1) / kWave, kScaleSlot = kScaleLoads * kWave * 16;
    static_assert(4 % KP == 0 || KP == 8, "whole stages of scales");
    static constexpr int kWeightsAt = SR * kRowSlot, kScalesAt = kWeightsAt + SW * kWeightSlot;
    template <bool FP8>
    static constexpr int bytes() { return kScalesAt + (FP8 ? SR * kScaleSlot : 0); }
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

// Of each expert of the call, in LDS: row tiles before it, first row, rows.
struct Experts {
    int base[kMaxExperts + 1];
    int first[kMaxExperts];
    int rows[kMaxExperts];
};

template <class T, bool GATED>
__device__ __forceinline__ Place place_of(const Product& P, const Experts& E, int X, int ntn, int t) {
    // the last expert with base[x] <= q: 16 at a time, then one by one
    const int q = t / ntn, lane = lane_id();
    int i = lane * 16;
    const int c = __popcll(ballot(i < X && E.base[i < X ? i : 0] <= q)) - 1;
    i = c * 16 + lane;
    const int x = c * 16 + __popcll(ballot(lane < 16 && i < X && E.base[i < X ? i : 0] <= q)) - 1;
    const int b0 = uniform(E.base[x]), mts = uniform(E.base[x + 1]) - b0;
    // row tiles in groups: within a group every row tile meets a weight tile before the next one
    // comes, so that both stay in the XCD's cache while its CUs use them
    const int in = t - b0 * ntn, g = in / (kGroupTiles * ntn), r = in - g * kGroupTiles * ntn;
    const int left = mts - g * kGroupTiles, gm = left < kGroupTiles ? left : kGroupTiles;
    Place p;
    p.cnt = uniform(E.rows[x]);
    // the expert's tiles share its rows evenly, in parts of 16
    const int rows = ((p.cnt + mts - 1) / mts + 15) & ~15;
    p.m0 = (g * kGroupTiles + r % gm) * rows;
    p.n0 = r / gm * (GATED ? T::BN / 2 : T::BN);
    p.end = p.m0 + rows < p.cnt ? p.m0 + rows : p.cnt;
    const int d = P.rb + x / P.L;
    p.e = (long)d * P.L + x % P.L;
    p.row0 = (long)d * P.B + uniform(E.first[x]);
    return p;
}

__device__ __forceinline__ void load_lds16(const void* src, uint8_t* dst) {
    __builtin_amdgcn_global_load_lds(src, (lds_void*)dst, 16, 0, 0);
}
__device__ __forceinline__ void load_lds4(const void* src, uint8_t* dst) {
    __builtin_amdgcn_global_load_lds(src, (lds_void*)dst, 4, 0, 0);
}

// A wave's loads of rows or of weights, stage after stage, tile after tile.  Lane l of a fill (8 rows of
// a step) lands at row l / 8, place l % 8, and fetches the row's 16-byte chunk (l % 8) ^ (l / 8): the reads
// of a 16-row part then spread over the LDS banks.  Rows past an expert's last repeat it; weight rows
// past the last repeat it too.  For the gated product the weight rows of a tile alternate, 16 gate rows
// and 16 up rows.
template <bool FP8, bool GATED, class T>
struct Loader {
    const uint8_t *from, *ups;  // the tile's first row, or its first weight row and up row
    uint32_t off[T::F];         // the lane's offset for each fill
    const float* scale[2];      // the lane's scales (e4m3, waves that load rows)
    int tile, k;                // next to load: stage k of a tile
    int slot, group;

    // Fill j of the wave's: fill i of the stage, its step and its first row.
    __device__ __forceinline__ static int fill(int j, bool rows) { return (uniform(wave_id()) & 3) * (rows ? T::FR : T::FW) + j; }

    __device__ __forceinline__ void aim(const Product& P, const Experts& E, int X, int ntn, bool rows) {
        const Place p = place_of<T, GATED>(P, E, X, ntn, tile);
        const int lane = lane_id();
        const int wrows = GATED ? 2 * P.C : P.C;
        const int chunk = (lane & 7) ^ (lane >> 3), r8 = lane >> 3;
        if (rows) {
            from = ups = P.a + (p.row0 + p.m0) * P.KB;
        } else {
            from = P.w + (p.e * wrows + p.n0) * P.KB;
            ups = from + (long)P.C * P.KB;
        }
        const int last = rows ? p.cnt - 1 - p.m0 : P.C - 1 - p.n0;
#pragma unroll
        for (int j = 0; j < T::F; ++j) {
            const int i = fill(j, rows), per = (rows ? T::BM : T::BN) / 8;
            const int kp = i / per, q = (i - kp * per) * 8;
            const int r = (!rows && GATED ? (q >> 5) * 16 + (q & 15) : q) + r8;
            off[j] = (uint32_t)(r < last ? r : last) * P.KB + kp * kStepBytes + chunk * 16;
        }
        if constexpr (FP8) {
            if (rows) {
                const int blocks = (wrows + 127) / 128;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int r = (uniform(wave_id()) + u * 4) * kWave + lane, j = r - T::BM;
                    const int m = r < last ? r : last;
                    int b = GATED ? (p.n0 + (j & 1) * P.C) / 128 : p.n0 / 128 + (j & 1);
                    b = b < blocks ? b : blocks - 1;
                    scale[u] = j < 0 || j > 1 ? P.as + (p.row0 + p.m0 + m) * P.KS : P.ws + (p.e * blocks + b) * P.KS;
                }
            }
        }
    }

    // Loads the next stage into the ring and moves on.
    __device__ __forceinline__ void load(const Product& P, const Experts& E, int X, int ntn, int tiles, int G, int stages,
                                         uint8_t* ring, bool rows) {
        const int lane = lane_id();
        const int kb = k * T::KP * kStepBytes;
        uint8_t* to = ring + (rows ? slot * T::kRowSlot : T::kWeightsAt + slot * T::kWeightSlot) + fill(0, rows) * 1024;
        if constexpr (FP8) {
            const int ks = k * T::KP;
            if (rows && ks % 4 == 0) {
                uint8_t* st = ring + T::kScalesAt + group * T::kScaleSlot;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int w = uniform(wave_id()) + u * 4;
                    if (u * 4 >= T::kScaleLoads || w >= T::kScaleLoads) break;
                    if (P.KS % 4 == 0) {  // 16-byte rows of scales
                        load_lds16(scale[u] + ks, st + w * 1024);
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            load_lds4(scale[u] + (ks + q < P.KS ? ks + q : P.KS - 1), st + (q * T::kScaleLoads + w) * 256);
                    }
                }
                group = group == T::SR - 1 ? 0 : group + 1;
            }
        }
        const uint8_t *f = from + kb, *v = ups + kb;
        const int mine = rows ? T::FR : T::FW, per = (rows ? T::BM : T::BN) / 8;
        if ((FP8 && T::KP == 1) || kb + T::KP * kStepBytes <= P.KB) {
#pragma unroll
            for (int j = 0; j < T::F; ++j) {
                const bool up = GATED && (fill(j, rows) % per) & 2;
                if (T::FR == T::FW || j < mine) load_lds16((up ? v : f) + off[j], to + j * 1024);
            }
        } else {  // the last stage of a row: zeros from the row's end on
            const int chunk = (lane & 7) ^ (lane >> 3);
#pragma unroll
            for (int j = 0; j < T::F; ++j) {
                const int i = fill(j, rows);
                const bool up = GATED && (i % per) & 2;
                uint32_t o = off[j];
                asm volatile("" : "+v"(o));  // keeps this path's addresses out of the other's registers
                const bool in = kb + i / per * kStepBytes + chunk * 16 < P.KB;
                if (T::FR == T::FW || j < mine) load_lds16(in ? (up ? v : f) + o : kZeros, to + j * 1024);
            }
        }
        slot = slot == (rows ? T::SR : T::SW) - 1 ? 0 : slot + 1;
        if (++k == stages) {
            k = 0;
            tile += G;
            if (tile < tiles) aim(P, E, X, ntn, rows);
        }
    }
};

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

// The block's tiles, v, v + G, ..., as one run of stages: the loads run ahead of the products, across
// the ends of tiles.
template <bool FP8, bool GATED, class T>
__device__ __forceinline__ void run_tiles(const Product& P, uint8_t* ring, const Experts& E, float* epi, int X, int v,
                                          int G) {
    static_assert(T::template bytes<FP8>() <= kRingBytes, "the ring");
    constexpr int MT = T::MT, NT = T::NT;
    const int ntn = (P.C + (GATED ? T::BN / 2 : T::BN) - 1) / (GATED ? T::BN / 2 : T::BN);
    const int tiles = E.base[X] * ntn;
    if (v >= tiles) return;
    const int stages = (P.KB + T::KP * kStepBytes - 1) / (T::KP * kStepBytes);
    const long total = (long)((tiles - 1 - v) / G + 1) * stages;
    const int lane = lane_id(), wave = uniform(wave_id());
    const bool rows = wave < T::WR, weights = wave >= kWaves - T::WW;
    const int lead = rows ? T::kRowLead : T::kWeightLead;
    Loader<FP8, GATED, T> L;
    L.tile = v;
    L.k = L.slot = L.group = 0;
    if (rows || weights) {
        L.aim(P, E, X, ntn, rows);
        for (int n = 0; n < lead && n < total; ++n) L.load(P, E, X, ntn, tiles, G, stages, ring, rows);
    }
    f32x4 acc[NT][MT];
    auto zero = [&] {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    };
    zero();
    const int r16 = lane & 15, g = lane >> 4;
    const int wm = wave / T::WN % T::WM, wn = wave % T::WN, kp = wave / (T::WM * T::WN);
    // row r's chunk c lies at place c ^ (r % 8); a lane takes chunks g and g + 4 of its row
    const int p0 = (g ^ (r16 & 7)) * 16, p1 = p0 ^ 64;
    const int at_a = (kp * T::BM + wm * 16 + r16) * kStepBytes;
    const int at_w = T::kWeightsAt + (kp * T::BN + wn * NT * 16 + r16) * kStepBytes;
    constexpr int kNext = T::WM * 16 * kStepBytes;  // to the wave's next 16 rows
    Place p = place_of<T, GATED>(P, E, X, ntn, v);
    int ct = v, ck = 0, rslot = 0, wslot = 0, group = -1;
    for (long n = 0; n < total; ++n) {
        if (rows) {
            if (n + T::kRowLead <= total) wait_loads<(T::kRowLead - 1) * T::FR>();
            else wait_loads<0>();
        } else if (weights) {
            if (n + T::kWeightLead <= total) wait_loads<(T::kWeightLead - 1) * T::FW>();
            else wait_loads<0>();
        }
        lds_barrier();
        const bool more = n + lead < total;
        if (more && (rows || (weights && !T::EARLY))) L.load(P, E, X, ntn, tiles, G, stages, ring, rows);
        const uint8_t* ta = ring + rslot * T::kRowSlot + at_a;
        const uint8_t* tw = ring + wslot * T::kWeightSlot + at_w;
        float sr[MT], sw[2];
        if constexpr (FP8) {
            const int ks = ck * T::KP;
            if (ks % 4 == 0) group = group == T::SR - 1 ? 0 : group + 1;
            // 16 bytes a row, or the four steps apart
            const bool by_row = P.KS % 4 == 0;
            const int one = by_row ? 4 : 1;
            const float* sc = (const float*)(ring + T::kScalesAt + group * T::kScaleSlot) +
                              (ks + kp) % 4 * (by_row ? 1 : T::kScaleLoads * kWave);
#pragma unroll
            for (int j = 0; j < MT; ++j) sr[j] = sc[((j * T::WM + wm) * 16 + r16) * one];
            sw[0] = sc[(T::BM + (GATED ? 0 : wn * NT * 16 / 128)) * one];
            sw[1] = GATED ? sc[(T::BM + 1) * one] : sw[0];
        }
        i32x4 w[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            w[i][0] = *(const i32x4*)(tw + i * 16 * kStepBytes + p0);
            w[i][1] = *(const i32x4*)(tw + i * 16 * kStepBytes + p1);
        }
        i32x4 b[2][2];
        b[0][0] = *(const i32x4*)(ta + p0);
        b[0][1] = *(const i32x4*)(ta + p1);
        if constexpr (T::EARLY) {
            lds_barrier();  // every wave has its weights
            if (more && weights) L.load(P, E, X, ntn, tiles, G, stages, ring, rows);
        }
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
                    const f32x4 q =
                        __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
                    const float s = sr[j] * sw[GATED ? (i & 1) : 0];
#pragma unroll
                    for (int u = 0; u < 4; ++u) acc[i][j][u] = __builtin_fmaf(q[u], s, acc[i][j][u]);
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
        rslot = rslot == T::SR - 1 ? 0 : rslot + 1;
        wslot = wslot == T::SW - 1 ? 0 : wslot + 1;
        if (++ck == stages) {
            write_tile<FP8, GATED, T>(P, p, acc, epi);
            zero();
            ck = 0;
            ct += G;
            if (ct < tiles) p = place_of<T, GATED>(P, E, X, ntn, ct);
        }
    }
    lds_barrier();
}

// The tiles, from few rows and columns to many.  The gated product needs two 16-row parts of a tile's
// weight rows in each wave (gate and up), and with e4m3 operands 256 of them in a tile: it quantises
// blocks of 128 output columns.
constexpr int kLevels = 4;
enum { kPlain, kGated, kWide };
template <int KIND, int I> struct TileOf;
template <> struct TileOf<kPlain, 0> { typedef Tile<16, 32, 1, 2, 4, 3, 7> type; };
template <> struct TileOf<kPlain, 1> { typedef Tile<32, 32, 1, 2, 4, 3, 5> type; };
template <> struct TileOf<kPlain, 2> { typedef Tile<16, 64, 1, 4, 2, 4, 7> type; };
template <> struct TileOf<kPlain, 3> { typedef Tile<32, 64, 1, 4, 2, 3, 7> type; };
template <> struct TileOf<kGated, 0> { typedef Tile<16, 32, 1, 1, 8, 2, 3> type; };
template <> struct TileOf<kGated, 1> { typedef Tile<32, 32, 2, 1, 4, 3, 5> type; };
template <> struct TileOf<kGated, 2> { typedef Tile<16, 64, 1, 2, 4, 3, 3> type; };
template <> struct TileOf<kGated, 3> { typedef Tile<32, 64, 2, 2, 2, 3, 7> type; };
template <int KIND> struct TileOf<KIND, 4> { typedef Tile<64, 64, 2, 2, 2, 3, 5> type; };
template <int KIND> struct TileOf<KIND, 5> { typedef Tile<64, 128, 2, 4, 1, 3, 7> type; };
template <int KIND> struct TileOf<KIND, 6> { typedef Tile<128, 128, 2, 4, 1, 3, 5> type; };
template <> struct TileOf<kWide, 3> { typedef Tile<16, 256, 1, 8, 1, 4, 4> type; };
template <> struct TileOf<kWide, 4> { typedef Tile<32, 256, 1, 8, 1, 3, 4> type; };
template <> struct TileOf<kWide, 5> { typedef Tile<64, 256, 1, 8, 1, 3, 3> type; };
template <int KIND> struct TileOf<KIND, 7> { typedef Tile<128, 256, 2, 4, 1, 2, 3> type; };
template <int KIND> struct TileOf<KIND, 8> { typedef Tile<160, 256, 2, 4, 1, 2, 2, true> type; };
template <int KIND> struct TileOf<KIND, 9> { typedef Tile<192, 256, 2, 4, 1, 2, 2, true> type; };
template <int KIND> struct TileOf<KIND, 10> { typedef Tile<256, 256, 2, 4, 1, 2, 2, true> type; };

// At each level an expert's rows make as few row tiles as fit `most` rows each (0: the largest tile;
// further levels smaller ones, for products that would leave CUs without a tile), and the tiles take
// the least height that holds their even share.
template <bool WIDE>
__device__ __forceinline__ int level_rows(int level) {
    return level == 0 ? 256 : level == 1 ? 128 : WIDE || level == 2 ? 64 : 32;
}
template <bool WIDE>
__device__ __forceinline__ int row_tiles(int rows, int level) {
    return (rows + level_rows<WIDE>(level) - 1) / level_rows<WIDE>(level);
}
template <bool WIDE>
__device__ __forceinline__ int tile_of(int rows, int level) {
    const int mts = row_tiles<WIDE>(rows, level), n = (rows + mts - 1) / (mts > 0 ? mts : 1);
    if (WIDE) return n > 192 ? 10 : n > 160 ? 9 : n > 128 ? 8 : n > 64 ? 7 : n > 32 ? 5 : n > 16 ? 4 : 3;
    if (level == 3) return n > 16 ? 1 : 0;
    if (n <= 32) return n > 16 ? 3 : 2;
    if (level == 2) return 4;
    if (n <= 64) return 5;
    return level == 1 ? 6 : n > 192 ? 10 : n > 160 ? 9 : n > 128 ? 8 : 7;
}

// Columns of weight rows of a tile, and the time of a step over K, in cycles.
template <bool WIDE>
__device__ __forceinline__ int tile_width(int i) {
    return WIDE || i >= 7 ? 256 : i >= 5 ? 128 : i >= 2 ? 64 : 32;
}
template <bool WIDE>
__device__ __forceinline__ int tile_time(int i, int rows) {
    return tile_width<WIDE>(i) * 4 + rows * tile_width<WIDE>(i) / 32 + 150;
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
    __shared__ Experts E;
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
        if (x < X) {
            rows[i] = expert_rows(P, x, &E.first[x]);
            E.rows[x] = rows[i];
        }
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
        scan_tiles<WIDE>(rows, level, i, X, E.base, part);
        int w = v - done % G;
        w = w < 0 ? w + G : w;
        run_tiles<FP8, GATED, T>(P, ring, E, epi, X, w, G);
        const int cols = GATED ? T::BN / 2 : T::BN;
        done += uniform(E.base[X]) * ((P.C + cols - 1) / cols);
    };
    run(typename TileOf<KIND, 10>::type(), 10);
    run(typename TileOf<KIND, 9>::type(), 9);
    run(typename TileOf<KIND, 8>::type(), 8);
    run(typename TileOf<KIND, 7>::type(), 7);
    if constexpr (!WIDE) run(typename TileOf<KIND, 6>::type(), 6);
    run(typename TileOf<KIND, 5>::type(), 5);
    run(typename TileOf<KIND, 4>::type(), 4);
    run(typename TileOf<KIND, 3>::type(), 3);
    if constexpr (!WIDE) {
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
