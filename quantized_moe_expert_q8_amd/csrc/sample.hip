// A token for each row of logits, from a given random number: temperature, top-k,
// top-p, min-p, and a draw in the order of the indexes.
//
// Weights e^((z - max) / T) are taken in 64 bits and summed as integers of 2^-S of
// the largest, S so that a row's sum stays below 2^63 (131072 tokens: 2^-46 each):
// sums are exact, whatever their order, so a token does not depend on how a row was
// split, and next to a border (u times the kept mass, p times the mass) the choice is
// that of the definition but for the weights' own roundings.
//
// The kept tokens are those above a threshold of the order-preserving keys, and of
// those equal to it the first few by index; a threshold is found by a radix
// selection, by count (top-k) or by mass (top-p), over few candidates:
//
//   k_scan   every segment of 512 logits: its largest key, and for rows that need it
//            the mass of all (over the segment's largest, since the row's is not known)
//   k_bins   rows whose candidates the largest keys do not narrow down: mass (and
//            count) by 1024 bins of a sixteenth of an octave below the row's largest
//   k_pick   a block a row: candidates, thresholds, the draw
//
// Candidates: for top-k the logits from the k-th largest of the segments' largest
// keys on, found in the k segments that have them; for min-p the segments whose
// largest passes it; else the bin that the threshold falls into.  Among bins the draw
// takes a tile of k_bins first, then a segment, then its logits in order; in a list it
// is one more selection, over the indexes.  A list that gets more candidates than LDS
// holds (a vocabulary in the order of its frequencies: the segments' largest say little)
// goes on by bins, which the row's block then makes itself (8 x 131072 f32, k = 50: 75
// us, by the whole row 270).  Rows with more than that in one bin (equal logits by the
// thousand; normal logits of a third of the temperature), with infinite logits, or of
// over 524288 logits go the slow way: selections over the whole row, 220 to 620 us for
// 131072 logits, since few digits take the additions of most logits.
//
// What bounds it: for few rows the chain of three launches and of a block's
// dependent steps (1 x 32000 f32 with top-k, and 5 x 131072 with top-p and min-p, 16
// us in a graph: 4 + 3 + 10), in which instructions that run once are fetched from memory: code
// that is not unrolled is faster here.  For many rows k_scan is bound by memory (256 x
// 131072 bf16 with top-k 13.9 us, 4.8 TB/s; 42 where every row needs its masses, by
// the arithmetic of 64 bits) and k_pick by what one CU issues for one row: 19 us with
// top-k = 50, 38 with rules of all kinds, 56 with top-p alone on normal logits.
#include "moeq8_cache.hpp"
#include "moeq8_lds.hpp"

namespace moeq8 {
namespace {

constexpr int SEG = 512;                          // logits a segment: 8 a lane
constexpr int MAX_SEGS = 1024;                    // more: the slow way
constexpr int BINS = 1024, PER_OCTAVE = 64;       // steps of the exponent's table; a bin is 4 of them
constexpr int CAP = 4096;                         // candidates that k_pick holds
constexpr int THREADS = 1024, WAVES = THREADS / 64;

struct SampleArgs {
    const void* z; int64_t z_stride;
    int64_t vocab;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t* top_k;
    int32_t* token;
    float* logprob;
    int bits;                                     // S
    uint32_t segs, tiles, tile_segs;              // tiles: of k_bins
    uint32_t* seg_top;                            // [rows][segs]
    uint64_t* seg_mass;                           // [rows][segs]
    uint64_t* bin_mass;                           // [rows][tiles][BINS]
    uint32_t* bin_count;                          // [rows][tiles][BINS]
};

// Keys of the logits in their order, equal for equal logits; 0 for what is never drawn.
__device__ __forceinline__ uint32_t key_of(float z) {
    const uint32_t b = __float_as_uint(z + 0.0f);
    const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return z > -__builtin_inff() ? k : 0u;        // false for NaN too
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float(key ^ (key >> 31 ? 0x80000000u : 0xffffffffu));
}
constexpr uint32_t KEY_INF = 0xff800000u, KEY_FIRST = 0x00800000u;       // of +inf and of the lowest finite logit

// A row's rules.
struct Rules {
    int64_t k;                                    // 0: all
    float p, least;                               // 1 and 0: all
    bool greedy;
    double per_logit;                             // steps of the exponent's table a logit: 64 log2(e) / T
    double per_nat;                               // 1 / T
    __device__ bool pure() const { return !greedy && !k && p == 1.0f && least == 0.0f; }
    // whether what min-p drops goes into the last bin (top-p counts it; not where top-p is
    // a part of what top-k leaves of it)
    __device__ bool rest() const { return least > 0.0f && !(k && p < 1.0f); }
    // whether k_scan sums the masses: for the draw, or for top-p beside min-p
    __device__ bool masses() const { return !greedy && !k && (p < 1.0f) == (least > 0.0f); }
};
__device__ __forceinline__ Rules rules_of(const SampleArgs& a, int64_t row) {
    Rules r;
    // a rule that is left out reads u's bits instead: loads under a branch each are
    // waited for one after another (what comes before a row's first decision took 5.7
    // us with them and a computed table of powers, and takes 1.5)
    const float* none = a.u;
    float t = (a.temperature ? a.temperature : none)[row], p = (a.top_p ? a.top_p : none)[row], least = (a.min_p ? a.min_p : none)[row];
    const int32_t k = (a.top_k ? a.top_k : (const int32_t*)none)[row];
    t = a.temperature ? t : 1.0f;
    r.greedy = !(t > 0.0f);
    r.k = a.top_k && k > 0 && k < a.vocab ? k : 0;
    r.p = a.top_p && p < 1.0f ? p : 1.0f;
    r.least = a.min_p && least > 0.0f ? fminf(least, 1.0f) : 0.0f;
    r.per_nat = 1.0 / (double)t;
    r.per_logit = (PER_OCTAVE * 1.4426950408889634) * r.per_nat;
    return r;
}

// Weights below a largest logit.  2^(t / 64) with t = i + r, i the nearest integer:
// 2^((i mod 64) / 64) from a table, 2^(r / 64) by its Taylor series, whose sixth term
// is below 2^-54.
struct Weigh {
    double top, c;                                // the largest logit; table steps a logit
    const double* table;                          // 2^(j / 64)
    // held where a weight is 0 in 64 bits, and not before: the plain draw takes weights as they are
    __device__ __forceinline__ double steps(float z) const { return fmax(((double)z - top) * c, -1100.0 * PER_OCTAVE); }
    __device__ __forceinline__ double at(double t, int& i) const {
        const double n = rint(t), x = (t - n) * (0.69314718055994531 / PER_OCTAVE);
        i = (int)n;
        double s = __builtin_fma(x, 1.0 / 120.0, 1.0 / 24.0);
        s = __builtin_fma(x, s, 1.0 / 6.0);
        s = __builtin_fma(x, s, 0.5);
        s = __builtin_fma(x, s, 1.0);
        const double e = table[i & (PER_OCTAVE - 1)];
        return __builtin_fma(x * s, e, e);        // times 2^(i >> 6)
    }
    __device__ __forceinline__ double real(float z) const {
        int i;
        const double v = at(steps(z), i);
        return __builtin_ldexp(v, i >> 6);
    }
    // in units of 2^-bits, bits <= 51: rounded by adding 2^52, whose low bits they then are
    static __device__ __forceinline__ uint64_t rounded(double v, int i, int bits) {
        return __builtin_bit_cast(uint64_t, __builtin_ldexp(v, (i >> 6) + bits) + 0x1p52) & ((1ull << 52) - 1);
    }
    __device__ __forceinline__ uint64_t units(float z, int bits) const {
        int i;
        const double v = at(steps(z), i);
        return rounded(v, i, bits);
    }
};
__device__ __forceinline__ int bin_of(int i) {    // i <= 0
    const int b = -i >> 2;
    return b < BINS ? b : BINS - 1;
}
__device__ __forceinline__ int bin_of(const Weigh& w, float z) { return bin_of((int)rint(w.steps(z))); }

// 2^(j / 64), correctly rounded.
__device__ const double POWERS[PER_OCTAVE] = {
    0x1.0000000000000p+0, 0x1.02c9a3e778061p+0, 0x1.059b0d3158574p+0, 0x1.0874518759bc8p+0,
    0x1.0b5586cf9890fp+0, 0x1.0e3ec32d3d1a2p+0, 0x1.11301d0125b51p+0, 0x1.1429aaea92de0p+0,
    0x1.172b83c7d517bp+0, 0x1.1a35beb6fcb75p+0, 0x1.1d4873168b9aap+0, 0x1.2063b88628cd6p+0,
    0x1.2387a6e756238p+0, 0x1.26b4565e27cddp+0, 0x1.29e9df51fdee1p+0, 0x1.2d285a6e4030bp+0,
    0x1.306fe0a31b715p+0, 0x1.33c08b26416ffp+0, 0x1.371a7373aa9cbp+0, 0x1.3a7db34e59ff7p+0,
    0x1.3dea64c123422p+0, 0x1.4160a21f72e2ap+0, 0x1.44e086061892dp+0, 0x1.486a2b5c13cd0p+0,
    0x1.4bfdad5362a27p+0, 0x1.4f9b2769d2ca7p+0, 0x1.5342b569d4f82p+0, 0x1.56f4736b527dap+0,
    0x1.5ab07dd485429p+0, 0x1.5e76f15ad2148p+0, 0x1.6247eb03a5585p+0, 0x1.6623882552225p+0,
    0x1.6a09e667f3bcdp+0, 0x1.6dfb23c651a2fp+0, 0x1.71f75e8ec5f74p+0, 0x1.75feb564267c9p+0,
    0x1.7a11473eb0187p+0, 0x1.7e2f336cf4e62p+0, 0x1.82589994cce13p+0, 0x1.868d99b4492edp+0,
    0x1.8ace5422aa0dbp+0, 0x1.8f1ae99157736p+0, 0x1.93737b0cdc5e5p+0, 0x1.97d829fde4e50p+0,
    0x1.9c49182a3f090p+0, 0x1.a0c667b5de565p+0, 0x1.a5503b23e255dp+0, 0x1.a9e6b5579fdbfp+0,
    0x1.ae89f995ad3adp+0, 0x1.b33a2b84f15fbp+0, 0x1.b7f76f2fb5e47p+0, 0x1.bcc1e904bc1d2p+0,
    0x1.c199bdd85529cp+0, 0x1.c67f12e57d14bp+0, 0x1.cb720dcef9069p+0, 0x1.d072d4a07897cp+0,
    0x1.d5818dcfba487p+0, 0x1.da9e603db3285p+0, 0x1.dfc97337b9b5fp+0, 0x1.e502ee78b3ff6p+0,
    0x1.ea4afa2a490dap+0, 0x1.efa1bee615a27p+0, 0x1.f50765b6e4540p+0, 0x1.fa7c1819e90d8p+0,
};
__device__ __forceinline__ void fill_table(double* table) {
    if (threadIdx.x < PER_OCTAVE) table[threadIdx.x] = POWERS[threadIdx.x];
}

// A lane's eight logits of segment `seg`, and the index of the first.  Where the row
// ends inside them they are its last eight, of which those of another lane are NaN,
// and past the row all are: loads without a branch, none of which waits for another.
template <typename T>
struct Eight {
    T raw[8];
    uint32_t first;
    __device__ __forceinline__ void load(const T* z, uint32_t seg, uint32_t vocab) {
        const uint32_t at = seg * SEG + (threadIdx.x & 63) * 8;
        first = at <= vocab - 8 ? at : vocab - 8;  // in bounds for any seg, whatever a shared workspace held
        if (vocab >= 8) {
            load_vec(raw, z + first);
        } else {
            first = at;
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) raw[j] = z[at + j < vocab ? at + j : 0];
        }
    }
    __device__ __forceinline__ void values(float (&v)[8], uint32_t seg, uint32_t vocab) const {
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) v[j] = to_f32(raw[j]);
        if ((seg + 1) * SEG > vocab) {
            const uint32_t at = seg * SEG + (threadIdx.x & 63) * 8;
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) v[j] = first + j >= at && first + j < vocab ? v[j] : __builtin_nanf("");
        }
    }
};

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = larger(v, moved<XOR1>(v));
    v = larger(v, moved<XOR2>(v));
    v = larger(v, moved<HALF_MIRROR>(v));
    v = larger(v, moved<MIRROR>(v));
    auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = larger(s[0], s[1]);
    s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return larger(s[0], s[1]);
}
__device__ __forceinline__ uint32_t wave_or(uint32_t v) {
    v |= moved<XOR1>(v);
    v |= moved<XOR2>(v);
    v |= moved<HALF_MIRROR>(v);
    v |= moved<MIRROR>(v);
    auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = s[0] | s[1];
    s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return s[0] | s[1];
}
__device__ __forceinline__ uint64_t wave_sum(uint64_t v) {
    v += moved<XOR1>(v);
    v += moved<XOR2>(v);
    v += moved<HALF_MIRROR>(v);
    v += moved<MIRROR>(v);
    auto cross = [](uint64_t x, bool halves) {
        const uint2 u = __builtin_bit_cast(uint2, x);
        if (halves) {
            const auto lo = __builtin_amdgcn_permlane32_swap(u.x, u.x, false, false), hi = __builtin_amdgcn_permlane32_swap(u.y, u.y, false, false);
            return __builtin_bit_cast(uint64_t, uint2{lo[0], hi[0]}) + __builtin_bit_cast(uint64_t, uint2{lo[1], hi[1]});
        }
        const auto lo = __builtin_amdgcn_permlane16_swap(u.x, u.x, false, false), hi = __builtin_amdgcn_permlane16_swap(u.y, u.y, false, false);
        return __builtin_bit_cast(uint64_t, uint2{lo[0], hi[0]}) + __builtin_bit_cast(uint64_t, uint2{lo[1], hi[1]});
    };
    return cross(cross(v, false), true);
}
// Sum over the lanes up to this one: within rows of 16 lanes, then over the rows.
template <int CTRL, int ROWS, typename V>
__device__ __forceinline__ V shifted(V v) {       // 0 where no lane is named
    const uint2 u = __builtin_bit_cast(uint2, v);
    return __builtin_bit_cast(V, uint2{(uint32_t)__builtin_amdgcn_update_dpp(0, (int)u.x, CTRL, ROWS, 0xf, false),
                                       (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u.y, CTRL, ROWS, 0xf, false)});
}
template <typename V>
__device__ __forceinline__ V row_scan(V v) {
    static_assert(sizeof(V) == 8, "two dwords");
    v += shifted<0x111, 0xf>(v);                  // row_shr 1, 2, 4, 8
    v += shifted<0x112, 0xf>(v);
    v += shifted<0x114, 0xf>(v);
    v += shifted<0x118, 0xf>(v);
    return v;
}
template <typename V>
__device__ __forceinline__ V wave_scan(V v) {
    v = row_scan(v);
    v += shifted<0x142, 0xa>(v);                  // the last lane of a row to the next one: rows 1 and 3
    v += shifted<0x143, 0xc>(v);                  // of the first two to the last two
    return v;
}
__device__ __forceinline__ uint32_t wave_scan32(uint32_t v) {
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false);
    return v;
}
template <typename V>
__device__ __forceinline__ V of_lane(V v, int lane) {
    const uint2 u = __builtin_bit_cast(uint2, v);
    return __builtin_bit_cast(V, uint2{(uint32_t)__builtin_amdgcn_readlane((int)u.x, lane), (uint32_t)__builtin_amdgcn_readlane((int)u.y, lane)});
}

// ---- segments --------------------------------------------------------------------

template <typename T, int PER>
__global__ __launch_bounds__(256) void k_scan(SampleArgs a, uint32_t blocks) {
    __shared__ double table[PER_OCTAVE];
    const uint32_t row = blockIdx.x / blocks, block = blockIdx.x - row * blocks;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const T* z = (const T*)a.z + row * a.z_stride;
    const uint32_t first = (block * 4 + wave) * PER, vocab = (uint32_t)a.vocab;
    Eight<T> e[PER];
#pragma unroll
    for (int s = 0; s < PER; ++s) e[s].load(z, first + s < a.segs ? first + s : a.segs - 1, vocab);
    const Rules r = rules_of(a, row);
    const bool masses = r.masses();
    if (masses) {
        fill_table(table);
        __syncthreads();
    }
#pragma unroll
    for (int s = 0; s < PER; ++s) {
        if (first + s >= a.segs) break;
        float v[8], most = -__builtin_inff();
        e[s].values(v, first + s, vocab);
#pragma unroll
        for (int j = 0; j < 8; ++j) most = fmaxf(most, v[j]);
        const uint32_t top = wave_max(key_of(most));
        uint64_t sum = 0;
        if (masses && top) {
            const Weigh w{(double)logit_of(top), r.per_logit, table};
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += v[j] > -__builtin_inff() ? w.units(v[j], 51) : 0;
            sum = wave_sum(sum);
        }
        if (lane == 0) {
            a.seg_top[(int64_t)row * a.segs + first + s] = top;
            if (masses) a.seg_mass[(int64_t)row * a.segs + first + s] = sum;
        }
    }
}

// ---- what k_bins and k_pick decide alike -------------------------------------------

enum Way { NONE, GREEDY, PURE, LIST, BY_BINS, SLOW };

struct Row {
    uint32_t key;                                 // largest key of segment threadIdx.x (blocks of MAX_SEGS threads)
    uint32_t top;                                 // of the row
    Way way;
};

// Needs 2 * N / 64 dwords of LDS; every thread of the block calls it.
template <int N>
__device__ __forceinline__ Row row_of(const SampleArgs& a, const Rules& r, int64_t row, uint32_t* lds, const double* table) {
    constexpr int PER = MAX_SEGS / N, W = N / 64;
    static_assert(W == 4 || W == 16, "lanes that have a wave's result each: a quad or a row");
    Row o;
    const uint32_t tid = threadIdx.x;
    uint32_t key[PER], most = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        key[i] = tid + i * N < a.segs ? a.seg_top[row * a.segs + tid + i * N] : 0u;
        most = larger(most, key[i]);
    }
    o.key = key[0];
    most = wave_max(most);
    if ((tid & 63) == 0) lds[tid >> 6] = most;
    __syncthreads();
    o.top = wave_max(lds[tid & (W - 1)]);
    // segments with a logit to draw, and those that pass min-p
    const Weigh w{(double)logit_of(o.top), r.per_logit, table};
    uint32_t counts = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool some = key[i] != 0, passes = some && o.top != KEY_INF && w.real(logit_of(key[i])) >= (double)r.least;
        counts += (uint32_t)__popcll(__ballot(some)) | (uint32_t)__popcll(__ballot(passes)) << 16;
    }
    if ((tid & 63) == 0) lds[W + (tid >> 6)] = counts;
    __syncthreads();
    counts = lds[W + (tid & (W - 1))];
    counts += moved<XOR1>(counts);
    counts += moved<XOR2>(counts);
    if constexpr (W == 16) {
        counts += moved<HALF_MIRROR>(counts);
        counts += moved<MIRROR>(counts);
    }
    const uint32_t segs = counts & 0xffffu, hits = counts >> 16;
    if (o.top == 0) o.way = NONE;
    else if (r.greedy) o.way = GREEDY;
    else if (o.top == KEY_INF) o.way = SLOW;
    else if (r.pure()) o.way = PURE;
    else if (segs <= CAP / SEG) o.way = LIST;
    // A list costs by its candidates, bins the same for all (8 x 131072 f32, 256 segments,
    // normal logits, list and bins: k = 20 19 and 32 us, 150 24 and 34, 250 40 and 36; 16 x
    // 32000, 63 segments, k = 60 21 and 29).  Of many segments a k near their number
    // would bring more candidates than the list holds.  Of min-p's candidates their number
    // is estimated from the segments without one, exp(-candidates / segments) of all;
    // up to 1024 make a list (min_p = 0.1 19 and 28 us, 0.05 25 and 28, 0.02 40 and 29; 64 x
    // 131072 bf16 24 and 54, 33 and 54, 56 and 54; 16 x 32000 14, 16 and 23 us, and 21).
    else if (r.k) o.way = r.k <= (segs <= 256 ? segs : segs * 3 / 4) ? LIST : BY_BINS;
    else if (r.least > 0.0f &&
             segs - hits + 0.5f >= segs * __expf(-1024.0f / segs)) o.way = LIST;
    else o.way = BY_BINS;
    return o;
}

// ---- bins --------------------------------------------------------------------------

// A wave's logits of a segment into the bins, but for those of the last bin that weigh
// nothing (-inf and NaN among them): no cut is made there, and logits masked with a
// finite value would take turns at it by the thousand (64 x 131072, k = 50 of 10000
// unmasked: 91 us by bins, and 45).
template <typename T>
__device__ __forceinline__ void add_to_bins(const SampleArgs& a, const Rules& r, const Weigh& w, const Eight<T>& e, uint32_t seg,
                                            unsigned long long* mass, uint32_t* count) {
    float v[8];
    e.values(v, seg, (uint32_t)a.vocab);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        int n;
        const double real = w.at(w.steps(v[j]), n);          // fmax takes a NaN for the least
        const uint64_t u = Weigh::rounded(real, n, a.bits);
        // what min-p drops counts for top-p, behind all others
        const int b = r.rest() && __builtin_ldexp(real, n >> 6) < (double)r.least ? BINS - 1 : bin_of(n);
        if (u == 0 && b == BINS - 1) continue;
        atomicAdd(&mass[b], (unsigned long long)u);
        if (r.k) atomicAdd(&count[b], 1u);
    }
}

template <typename T>
__global__ __launch_bounds__(256) void k_bins(SampleArgs a) {
    __shared__ double table[PER_OCTAVE];
    __shared__ uint32_t words[8];
    __shared__ unsigned long long mass[BINS];
    __shared__ uint32_t count[BINS];
    const uint32_t row = blockIdx.x / a.tiles, tile = blockIdx.x - row * a.tiles, tid = threadIdx.x;
    const Rules r = rules_of(a, row);
    if (r.greedy || r.pure()) return;
    fill_table(table);
    __syncthreads();
    const Row o = row_of<256>(a, r, row, words, table);
    if (o.way != BY_BINS) return;
#pragma unroll
    for (int i = 0; i < BINS; i += 256) mass[tid + i] = count[tid + i] = 0;
    __syncthreads();
    const Weigh w{(double)logit_of(o.top), r.per_logit, table};
    const T* z = (const T*)a.z + row * a.z_stride;
    const uint32_t first = tile * a.tile_segs, last = first + a.tile_segs < a.segs ? first + a.tile_segs : a.segs;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6), vocab = (uint32_t)a.vocab;
    constexpr uint32_t AHEAD = 4;
#pragma unroll 1
    for (uint32_t seg = first + wave; seg < last; seg += 4 * AHEAD) {
        Eight<T> e[AHEAD];
#pragma unroll
        for (uint32_t i = 0; i < AHEAD; ++i) e[i].load(z, seg + 4 * i < last ? seg + 4 * i : seg, vocab);
#pragma unroll
        for (uint32_t i = 0; i < AHEAD; ++i) {
            if (seg + 4 * i >= last) break;
            add_to_bins(a, r, w, e[i], seg + 4 * i, mass, count);
        }
    }
    __syncthreads();
    const int64_t at = ((int64_t)row * a.tiles + tile) * BINS + tid;
#pragma unroll
    for (int i = 0; i < BINS; i += 256) {
        a.bin_mass[at + i] = mass[tid + i];
        if (r.k) a.bin_count[at + i] = count[tid + i];
    }
}

// ---- the pick ------------------------------------------------------------------------

struct Lds {
    double table[PER_OCTAVE];
    uint64_t hist[256];
    uint64_t sums[WAVES];
    uint64_t rest, pick_before;
    uint32_t words[2 * WAVES];
    uint32_t pick_key, n, seg, hits, from, least;
    uint64_t seg_sum[64];
    uint32_t top[MAX_SEGS];                       // the segments' largest keys
    uint16_t hit[MAX_SEGS];
    uint64_t weight[CAP];
    uint32_t key[CAP], index[CAP];
};

// Sum over the threads before this one, and over all.
template <typename V>
__device__ __forceinline__ V block_scan(V v, Lds& s, V& all) {
    const V up_to = wave_scan(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 63) s.sums[threadIdx.x >> 6] = __builtin_bit_cast(uint64_t, up_to);
    __syncthreads();
    static_assert(WAVES == 16, "a row of lanes");
    const V waves = row_scan(__builtin_bit_cast(V, s.sums[threadIdx.x & 15]));
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    all = of_lane(waves, 15);
    return (wave ? of_lane(waves, wave - 1) : (V)0) + (up_to - v);
}
__device__ __forceinline__ uint64_t block_sum(uint64_t v, Lds& s) {
    uint64_t all;
    block_scan(v, s, all);
    return all;
}

__device__ __forceinline__ void wave_order() {    // this wave's LDS operations before are seen by those after
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
// By one wave: the digit up to which, from 255 down, there is `want` in s.hist (or 0);
// `before`, what is before s.hist's, grows by what is before the digit.
__device__ __forceinline__ uint32_t digit_reaching(Lds& s, uint64_t want, uint64_t& before) {
    const uint32_t lane = threadIdx.x & 63;       // lane l has the four digits from 255 - 4 l down
    uint64_t h[4], sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) sum += h[j] = s.hist[255 - 4 * lane - j];
    uint64_t at = before + wave_scan(sum) - sum;
    const uint64_t reach = __ballot(at + sum >= want);
    const int from = reach ? (int)__builtin_ctzll(reach) : 63;
    int digit = 0;
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (digit == j && at + h[j] < want) {
            at += h[j];
            digit = j + 1;
        }
    before = of_lane(at, from);
    return (uint32_t)(255 - 4 * from - __builtin_amdgcn_readlane(digit, from));
}

// The key from which on, in falling order, the sum reaches `want` (or the last one),
// and the sum before it.  each(f) calls f(key, amount) for this thread's part.  Only
// the bits in which the keys differ are gone through: a list's share most upper ones.
template <typename E>
__device__ __forceinline__ uint32_t select(Lds& s, uint64_t want, uint64_t& before, E each) {
    const uint32_t wave = threadIdx.x >> 6;
    uint32_t any = 0, all = ~0u;
    each([&](uint32_t key, uint64_t) {
        any |= key;
        all &= key;
    });
    any = wave_or(any);
    all = wave_or(~all);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        s.words[wave] = any;
        s.words[WAVES + wave] = all;
    }
    __syncthreads();
    any = wave_or(s.words[threadIdx.x & (WAVES - 1)]);
    all = ~wave_or(s.words[WAVES + (threadIdx.x & (WAVES - 1))]);
    int left = 32 - __builtin_clz((any & ~all) | 1u);            // bits still open
    uint32_t prefix = (uint32_t)((uint64_t)all >> left << left);
    before = 0;
#pragma unroll 1
    while (left > 0) {
        const int from = left > 8 ? left - 8 : 0;
        if (threadIdx.x < 256) s.hist[threadIdx.x] = 0;
        __syncthreads();
        each([&](uint32_t key, uint64_t amount) {
            if ((uint64_t)(key ^ prefix) >> left == 0)
                atomicAdd((unsigned long long*)&s.hist[key >> from & 255], (unsigned long long)amount);
        });
        __syncthreads();
        if (wave == 0) {
            uint64_t at = before;
            const uint32_t digit = digit_reaching(s, want, at);
            if (threadIdx.x == 0) {
                s.pick_key = prefix | digit << from;
                s.pick_before = at;
            }
        }
        __syncthreads();
        prefix = s.pick_key;
        before = s.pick_before;
        left = from;
    }
    return prefix;
}

// The same by one wave, which needs no barriers: for lists of a few hundred.
template <typename E>
__device__ __forceinline__ uint32_t wave_select(Lds& s, uint64_t want, uint64_t& before, E each) {
    const uint32_t lane = threadIdx.x & 63;
    // only the bits that differ: the keys of a list share most of the upper ones
    uint32_t any = 0, all = ~0u;
    each([&](uint32_t key, uint64_t) {
        any |= key;
        all &= key;
    });
    any = wave_or(any);
    all = ~wave_or(~all);
    int left = 32 - __builtin_clz((any & ~all) | 1u);            // bits still open
    uint32_t prefix = (uint32_t)((uint64_t)all >> left << left);
    before = 0;
#pragma unroll 1
    while (left > 0) {
        const int from = left > 8 ? left - 8 : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) s.hist[lane + 64 * j] = 0;
        wave_order();
        each([&](uint32_t key, uint64_t amount) {
            if ((uint64_t)(key ^ prefix) >> left == 0)
                atomicAdd((unsigned long long*)&s.hist[key >> from & 255], (unsigned long long)amount);
        });
        wave_order();
        prefix |= digit_reaching(s, want, before) << from;
        wave_order();
        left = from;
    }
    return prefix;
}

__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
    for (int i = 32; i; i >>= 1) {
        const uint64_t t = __shfl_xor((unsigned long long)v, i);
        v = t > v ? t : v;
    }
    return v;
}

// By one wave: the token of a segment, the first in order up to which there is more
// than `rest` (the last one with a weight, where roundings left none).
template <typename T, typename D>
__device__ __forceinline__ void pick_in_segment(const SampleArgs& a, const Rules& r, int64_t row, const T* z, uint32_t seg, uint64_t rest,
                                double top, double mass, D drawn) {
    const uint32_t lane = threadIdx.x & 63;
    Eight<T> e;
    float v[8];
    e.load(z, seg, (uint32_t)a.vocab);
    e.values(v, seg, (uint32_t)a.vocab);
    uint64_t u[8], sum = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += u[j] = drawn(v[j], e.first + j);
    uint64_t at = wave_scan(sum) - sum;
    const uint64_t past = __ballot(at + sum > rest), any = __ballot(sum > 0);
    const uint32_t has = past ? (uint32_t)__builtin_ctzll(past) : 63u - (uint32_t)__builtin_clzll(any);
    if (lane != has) return;
    int pick = 0;
    float value = 0.0f;
    bool done = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (u[j] && !done) {
            pick = j;
            value = v[j];
        }
        at += u[j];
        done |= at > rest;
    }
    a.token[row] = (int32_t)(e.first + pick);
    if (a.logprob) a.logprob[row] = (float)(((double)value - top) * r.per_nat - log(mass));
}

// False, with nothing written, for a row that has to go the slow way.
template <typename T>
__device__ __forceinline__ bool pick_fast(const SampleArgs& a, const Rules& r, int64_t row, Lds& s) {
    const T* z = (const T*)a.z + row * a.z_stride;
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), vocab = (uint32_t)a.vocab;
    const Row o = row_of<THREADS>(a, r, row, s.words, s.table);
    if (o.way == NONE) {
        if (tid == 0) {
            a.token[row] = -1;
            if (a.logprob) a.logprob[row] = -__builtin_inff();
        }
        return true;
    }
    if (o.way == SLOW) return false;
    const float top = logit_of(o.top);
    const Weigh w{(double)top, r.per_logit, s.table};

    // ---- greedy: the first of the largest ----
    if (o.way == GREEDY) {
        if (tid == 0) s.seg = ~0u;
        __syncthreads();
        if (o.key == o.top) atomicMin(&s.seg, tid);
        __syncthreads();
        if (wave == 0) {
            Eight<T> e;
            float v[8];
            e.load(z, s.seg, vocab);
            e.values(v, s.seg, vocab);
            uint32_t at = ~0u;
#pragma unroll
            for (int j = 7; j >= 0; --j)
                if (v[j] == logit_of(o.top)) at = e.first + j;
            const uint64_t has = __ballot(at != ~0u);
            if (lane == (uint32_t)__builtin_ctzll(has)) {
                a.token[row] = (int32_t)at;
                if (a.logprob) a.logprob[row] = 0.0f;
            }
        }
        return true;
    }

    float uf = a.u[row];
    if (!(uf > 0.0f)) uf = 0.0f;

    if (o.way == PURE) {
        const double factor = o.key ? w.real(logit_of(o.key)) : 0.0;
        const double mine = o.key ? (double)a.seg_mass[row * a.segs + tid] * 0x1p-51 * factor : 0.0;
        double all;
        const double before = block_scan(mine, s, all), target = (double)uf * all;
        if (tid == 0) s.seg = ~0u;
        __syncthreads();
        // the first segment up to which there is more than the target; at the end of
        // the mass the last one with any
        const bool holds = mine > 0.0 && before + mine > target;
        if (holds) atomicMin(&s.seg, tid);
        __syncthreads();
        uint32_t seg = s.seg;
        if (seg == ~0u) {
            __syncthreads();
            if (tid == 0) s.seg = 0;
            __syncthreads();
            if (mine > 0.0) atomicMax(&s.seg, tid);
            __syncthreads();
            seg = s.seg;
        }
        if (tid == seg) {
            const double rest = (target - before) / factor * 0x1p51;
            s.rest = rest > 0.0 ? (uint64_t)fmin(rest, 0x1p61) : 0;
            s.pick_key = o.key;
        }
        __syncthreads();
        if (wave == 0) {
            const Weigh own{(double)logit_of(s.pick_key), w.c, s.table};
            pick_in_segment(a, r, row, z, seg, s.rest, (double)top, all,
                            [&](float v, uint32_t) { return v > -__builtin_inff() ? own.units(v, 51) : 0; });
        }
        return true;
    }

    // By a wave: the smallest key with pass, which larger ones have too, near the logit
    // `guess`: 64 keys there at once, or else a search of 6 steps.
    auto first_key = [&](double guess, auto pass) {
        const float near = (float)guess;
        const uint32_t mid = near > -__FLT_MAX__ ? key_of(near) : KEY_FIRST + 32, at0 = (mid < KEY_FIRST + 32 ? KEY_FIRST + 32 : mid) - 32 + lane;
        const uint64_t in = __ballot(at0 >= o.top || pass(logit_of(at0)));
        if (in && !(in & 1)) return (uint32_t)__builtin_amdgcn_readlane((int)at0, (int)__builtin_ctzll(in));
        uint32_t lo = KEY_FIRST - 1, hi = o.top;
#pragma unroll 1
        while (hi - lo > 1) {
            const uint32_t step = (hi - lo + 63) / 64, at = hi - lo > step * (lane + 1) ? lo + step * (lane + 1) : hi;
            const int first = __builtin_ctzll(__ballot(at == hi || pass(logit_of(at))));
            hi = (uint32_t)__builtin_amdgcn_readlane((int)at, first);
            lo = first ? (uint32_t)__builtin_amdgcn_readlane((int)at, first - 1) : lo;
        }
        return hi;
    };
    s.top[tid] = o.key;
    if (wave == 0) {
        const uint32_t least = r.least > 0.0f ? first_key((double)top + log((double)r.least) / r.per_nat, [&](float v) { return w.real(v) >= (double)r.least; }) : KEY_FIRST;
        if (lane == 0) s.least = least;
    }

    // The segments with keys from lo on, in order; every thread calls it.
    auto hit_segments = [&](uint32_t lo) {
        if (wave == 0) {
            uint32_t hits = 0;
#pragma unroll 1
            for (uint32_t from = 0; from < a.segs; from += 64) {
                const bool hit = from + lane < a.segs && s.top[from + lane] >= lo;
                const uint64_t all = __ballot(hit);
                if (hit)
                    s.hit[hits + __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0))] = (uint16_t)(from + lane);
                hits += (uint32_t)__popcll(all);
            }
            if (lane == 0) {
                s.hits = hits;
                s.n = 0;
            }
        }
        __syncthreads();
    };
    // Candidates: the keys from lo to below hi into the list, with their weights; their
    // order there does not matter.  False if they are too many.
    auto gather = [&](uint32_t lo, uint32_t hi) {
        hit_segments(lo);
        const uint32_t hits = s.hits;
        const float least = logit_of(lo), past = logit_of(hi);
        constexpr uint32_t AHEAD = 4;
#pragma unroll 1
        for (uint32_t h = wave; h < hits; h += WAVES * AHEAD) {
            Eight<T> e[AHEAD];
            uint32_t seg[AHEAD];
#pragma unroll
            for (uint32_t i = 0; i < AHEAD; ++i) {
                seg[i] = __builtin_amdgcn_readfirstlane(s.hit[h + i * WAVES < hits ? h + i * WAVES : h]);
                e[i].load(z, seg[i], vocab);
            }
            // A bit for each of the lane's candidates.  These are few and far between:
            // each lane writes its own, and what is written is the index alone.
            uint32_t in = 0;
#pragma unroll
            for (uint32_t i = 0; i < AHEAD; ++i) {
                float v[8];
                e[i].values(v, seg[i], vocab);
                if (h + i * WAVES >= hits) break;
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) in |= v[j] >= least && v[j] < past ? 1u << (8 * i + j) : 0u;
            }
            if (!__any(in)) continue;
            const uint32_t mine = (uint32_t)__builtin_popcount(in), up_to = wave_scan32(mine);
            uint32_t at = 0;
            if (lane == 63) at = atomicAdd(&s.n, up_to);
            at = (uint32_t)__builtin_amdgcn_readlane((int)at, 63) + up_to - mine;
            for (; in; in &= in - 1, ++at) {
                const uint32_t b = (uint32_t)__builtin_ctz(in), i = b / 8;
                static_assert(AHEAD == 4, "the choice below");
                const uint32_t first = i < 2 ? (i == 0 ? e[0].first : e[1].first) : (i == 2 ? e[2].first : e[3].first);
                if (at < CAP) s.index[at] = first + b % 8;
            }
        }
        __syncthreads();
        const uint32_t n = s.n;
        if (n > CAP) return false;
#pragma unroll 1
        for (uint32_t e = tid; e < n; e += THREADS) {
            const float v = to_f32(z[s.index[e]]);
            s.key[e] = key_of(v);
            s.weight[e] = w.units(v, a.bits);
        }
        __syncthreads();
        return true;
    };

    // ---- wave 0's work on the list ----
    auto listed = [&](auto f) {                   // four entries' loads at a time
        const uint32_t n = s.n;
#pragma unroll 1
        for (uint32_t e = lane; e < n; e += 256) {
            uint32_t key[4], index[4];
            uint64_t u[4];
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                const uint32_t at = e + 64 * i < n ? e + 64 * i : e;
                key[i] = s.key[at];
                index[i] = s.index[at];
                u[i] = s.weight[at];
            }
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i)
                if (e + 64 * i < n) f(key[i], index[i], u[i]);
        }
    };
    // the threshold that `count` keys are at or above
    auto cut_by_count = [&](uint64_t count, uint32_t& floor, uint64_t& ties, uint64_t above = 0) {
        uint64_t before;
        floor = wave_select(s, count - above, before, [&](auto add) { listed([&](uint32_t key, uint32_t, uint64_t) { add(key, 1); }); });
        ties = count - above - before;
    };
    // the mass above `floor`, how many keys are equal to it, and the weight of each
    auto mass_of = [&](uint32_t floor, uint64_t& equal, uint64_t& unit) {
        uint64_t sum = 0;
        uint32_t n = 0;
        unit = 0;
        listed([&](uint32_t key, uint32_t, uint64_t u) {
            sum += key > floor ? u : 0;
            unit = key == floor ? u : unit;
            n += key == floor;
        });
        unit = wave_max64(unit);
        equal = of_lane((uint64_t)wave_scan32(n), 63);
        return wave_sum(sum);
    };
    // of the listed keys above `floor`, and `ties` of those equal to it (of weight
    // `unit`), those before which there is less than `want` of mass
    auto cut_by_mass = [&](uint64_t want, uint32_t& floor, uint64_t& ties, uint64_t unit) {
        uint64_t before, equal;
        const uint32_t key = wave_select(s, want, before, [&](auto add) {
            listed([&](uint32_t key, uint32_t, uint64_t u) { if (key > floor) add(key, u); });
            if (unit && lane == 0) add(floor, ties * unit);
        });
        mass_of(key, equal, unit);
        const uint64_t n = unit ? (want - before + unit - 1) / unit : ~0ull;
        ties = key == floor && ties < n ? ties : n;
        floor = key;
    };
    auto part_of = [&](uint64_t all) {            // top-p's
        const uint64_t want = (uint64_t)ceil(fmax(r.p, 0.0f) * (double)all);
        return want < 1 ? (uint64_t)1 : want;
    };
    // the index of the last of the ties (all keys equal to the threshold are listed)
    auto last_tie = [&](uint32_t floor, uint64_t ties, uint64_t equal) -> uint32_t {
        uint64_t before;
        if (ties >= equal) return vocab;
        return 0xffffffu - wave_select(s, ties, before, [&](auto add) {
            listed([&](uint32_t key, uint32_t i, uint64_t) { if (key == floor) add(0xffffffu - i, 1); });
        });
    };

    if (o.way == LIST) {
        const bool by_least = !r.k && r.least > 0.0f;
        double all = 0.0;
        if (by_least && r.p < 1.0f)               // top-p is a part of all logits, not of the list
            block_scan(o.key ? (double)a.seg_mass[row * a.segs + tid] * 0x1p-51 * w.real(logit_of(o.key)) : 0.0, s, all);
        __syncthreads();
        if (r.k && wave == 0) {
            // the k-th largest; where fewer segments than k have a logit all of their logits
            uint64_t before;
            uint32_t some = 0;
            auto tops = [&](auto f) {
#pragma unroll 1
                for (uint32_t e = lane; e < a.segs; e += 256) {
                    uint32_t key[4];
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i) key[i] = s.top[e + 64 * i < a.segs ? e + 64 * i : e];
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i)
                        if (e + 64 * i < a.segs && key[i]) f(key[i]);
                }
            };
            tops([&](uint32_t) { ++some; });
            uint32_t from = KEY_FIRST;
            if (of_lane((uint64_t)wave_scan32(some), 63) >= (uint64_t)r.k)
                from = wave_select(s, (uint64_t)r.k, before, [&](auto add) { tops([&](uint32_t key) { add(key, 1); }); });
            // logits that weigh nothing, masked with a finite value say, need not be there
            if (bin_of(w, logit_of(from)) == BINS - 1)
                from = first_key((double)top - (4.0 * BINS - 4.5) / w.c, [&](float v) { return bin_of(w, v) < BINS - 1; });
            if (lane == 0) s.from = from;
        }
        __syncthreads();
        if (gather(r.k ? s.from : s.least, KEY_INF)) {
            if (wave != 0) return true;
            uint32_t floor = 0;
            uint64_t ties = ~0ull, before, unit, equal;
            if (r.k && (uint64_t)r.k < s.n) cut_by_count((uint64_t)r.k, floor, ties);
            if (r.p < 1.0f) {
                uint64_t have = mass_of(floor, equal, unit);
                have += unit ? ties * unit : 0;
                const uint64_t want = part_of(by_least ? (uint64_t)rint(__builtin_ldexp(all, a.bits)) : have);
                if (have >= want) cut_by_mass(want, floor, ties, unit);       // else min-p cuts above top-p
            }
            uint32_t limit = vocab;
            if (floor) {
                mass_of(floor, equal, unit);
                limit = last_tie(floor, ties, equal);
            }
            // the draw: by index, the first up to which there is more than the target
            const uint32_t least = s.least;
            auto drawn = [&](uint32_t key, uint32_t i, uint64_t u) { return key >= least && (key > floor || (key == floor && i <= limit)) ? u : 0; };
            uint64_t total = 0;
            listed([&](uint32_t key, uint32_t i, uint64_t u) { total += drawn(key, i, u); });
            total = wave_sum(total);
            uint64_t target = (uint64_t)((double)uf * (double)total);
            if (target >= total) target = total - 1;
            uint32_t token = 0xffffffu - wave_select(s, target + 1, before, [&](auto add) {
                listed([&](uint32_t key, uint32_t i, uint64_t u) {
                    const uint64_t d = drawn(key, i, u);
                    if (d) add(0xffffffu - i, d);
                });
            });
            token = token < vocab ? token : vocab - 1;
            if (lane == 0) {
                a.token[row] = (int32_t)token;
                if (a.logprob)
                    a.logprob[row] = (float)(((double)to_f32(z[token]) - (double)top) * r.per_nat - log(__builtin_ldexp((double)total, -a.bits)));
            }
            return true;
        }
        // more than the list holds: on by bins, which k_bins has not made
        static_assert(THREADS == BINS && CAP >= BINS, "a thread a bin, in the list's place");
        unsigned long long* const mass = (unsigned long long*)s.weight;
#pragma unroll 1
        for (uint32_t t = 0; t < a.tiles; ++t) {
            mass[tid] = s.key[tid] = 0;
            __syncthreads();
            const uint32_t first = t * a.tile_segs, last = first + a.tile_segs < a.segs ? first + a.tile_segs : a.segs;
#pragma unroll 1
            for (uint32_t seg = first + wave; seg < last; seg += WAVES) {
                Eight<T> e;
                e.load(z, seg, vocab);
                add_to_bins(a, r, w, e, seg, mass, s.key);
            }
            __syncthreads();
            a.bin_mass[(row * a.tiles + t) * BINS + tid] = mass[tid];
            if (r.k) a.bin_count[(row * a.tiles + t) * BINS + tid] = s.key[tid];
        }
        __syncthreads();
    }

    // ---- by bins: thread b has bin b ----
    uint64_t bin_mass = 0, bin_count = 0;
#pragma unroll 4
    for (uint32_t t = 0; t < a.tiles; ++t) {
        bin_mass += a.bin_mass[(row * a.tiles + t) * BINS + tid];
        if (r.k) bin_count += a.bin_count[(row * a.tiles + t) * BINS + tid];
    }
    uint32_t held = ~0u;                          // the bin in the list
    uint32_t floor = 0, limit = vocab;
    uint64_t ties = ~0ull, unit = 0;              // of the keys equal to `floor`, and the weight of each
    auto shared = [&](auto f) {                   // the list by the block: here it has up to thousands
#pragma unroll 1
        for (uint32_t e = tid; e < s.n; e += THREADS) f(s.key[e], s.index[e], s.weight[e]);
    };
    if (tid == 0) s.n = 0;
    // top-k by the counts, then top-p by the masses, then min-p, whose bin the list has
    // to hold unless what it drops is in the last bin
#pragma unroll 1
    for (int step = 0; step < 3; ++step) {
        if (step == 0 ? r.k == 0 : step == 1 ? r.p == 1.0f : r.least == 0.0f || r.rest()) continue;
        uint64_t want = 0, before = 0;
        uint32_t bin;
        if (step < 2) {
            const uint64_t amount = step ? bin_mass : bin_count;
            uint64_t all;
            const uint64_t at = block_scan(amount, s, all);
            if (!step && (uint64_t)r.k >= all) continue;
            want = step ? part_of(all) : (uint64_t)r.k;
            if (at < want && at + amount >= want) {
                s.seg = tid;
                s.rest = at;
            }
            __syncthreads();
            bin = s.seg;
            before = s.rest;
            if (bin == BINS - 1) continue;        // min-p cuts above, or what is cut there weighs nothing
        } else {
            __syncthreads();
            if (s.least <= floor) continue;       // the others cut above
            bin = (uint32_t)bin_of(w, logit_of(s.least));
            if (bin == BINS - 1) continue;
        }
        if (bin != held) {
            if (wave == 0) {
                // a bin has 4 steps, rounded to the nearest: from 4 bin + 3.5 to 4 bin - 0.5 below
                const uint32_t lo = first_key((double)top - (4.0 * bin + 3.5) / w.c, [&](float v) { return bin_of(w, v) <= (int)bin; });
                const uint32_t hi = bin ? first_key((double)top - (4.0 * bin - 0.5) / w.c, [&](float v) { return bin_of(w, v) < (int)bin; }) : KEY_INF;
                if (lane == 0) {
                    s.from = lo;
                    s.pick_key = hi;
                }
            }
            __syncthreads();
            if (!gather(s.from, s.pick_key)) return false;
        }
        const uint32_t old = bin == held ? floor : 0;
        const uint64_t old_ties = ties, old_unit = bin == held ? unit : 0;
        uint64_t in_bin;
        if (step == 0) {
            floor = select(s, want - before, in_bin, [&](auto add) { shared([&](uint32_t key, uint32_t, uint64_t) { add(key, 1); }); });
            ties = want - before - in_bin;
        } else if (step == 1) {
            floor = select(s, want - before, in_bin, [&](auto add) {
                shared([&](uint32_t key, uint32_t, uint64_t u) { if (key > old) add(key, u); });
                if (old_unit && tid == 0) add(old, old_ties * old_unit);
            });
        } else {
            floor = s.least;                      // all that are equal to it
            ties = ~0ull;
        }
        uint64_t mass = 0, equal = 0;
        shared([&](uint32_t key, uint32_t, uint64_t u) {
            mass += key > floor ? u : 0;
            equal += key == floor;
        });
        mass = block_sum(mass, s);
        equal = block_sum(equal, s);
        unit = equal ? w.units(logit_of(floor), a.bits) : 0;
        if (step == 1) {
            const uint64_t n = unit ? (want - before - in_bin + unit - 1) / unit : ~0ull;
            ties = floor == old && old_ties < n ? old_ties : n;
        }
        limit = vocab;
        if (ties < equal) {
            uint64_t none;
            limit = 0xffffffu - select(s, ties, none, [&](auto add) {
                shared([&](uint32_t key, uint32_t i, uint64_t) { if (key == floor) add(0xffffffu - i, 1); });
            });
        } else {
            ties = equal;
        }
        __syncthreads();
        held = bin;
        const uint64_t left = mass + ties * unit;
        // the bins' masses without what is dropped
        bin_mass = tid < bin ? bin_mass : (tid == bin ? left : 0);
    }
    __syncthreads();
    // where min-p cuts above the others: all that are equal to its key, of the bins all but the last
    const bool by_least = r.rest() && s.least > floor;
    if (by_least) {
        floor = s.least;
        limit = vocab;
        held = BINS - 1;
    }
    const float above = floor ? logit_of(floor) : -__builtin_inff();
    auto drawn = [&](float v, uint32_t i) -> uint64_t {
        return v > above || (floor && v == above && i <= limit) ? w.units(v, a.bits) : 0;
    };
    // ---- the kept mass by tiles, a wave each: of the bins above the held one as they are,
    // of that one by the list; then by the segments of the tile that the draw falls into,
    // and in the segment ----
    static_assert(WAVES == 16, "a wave a tile");
    if (wave < a.tiles) {
        uint64_t sum = 0;
#pragma unroll 4
        for (uint32_t b = lane; b < BINS; b += 64) sum += b < held ? a.bin_mass[(row * a.tiles + wave) * BINS + b] : 0;
        const uint32_t n = held == ~0u || by_least ? 0 : s.n, first = wave * a.tile_segs * SEG, past = first + a.tile_segs * SEG;
#pragma unroll 4
        for (uint32_t e = lane; e < n; e += 64) {
            const uint32_t key = s.key[e], i = s.index[e];
            if (i >= first && i < past && (key > floor || (key == floor && i <= limit))) sum += s.weight[e];
        }
        sum = wave_sum(sum);
        if (lane == 0) s.seg_sum[wave] = sum;
    }
    __syncthreads();
    const uint64_t tile_mass = lane < a.tiles ? s.seg_sum[lane] : 0, tile_upto = wave_scan(tile_mass), all = of_lane(tile_upto, 63);
    uint64_t target = (uint64_t)((double)uf * (double)all);
    if (target >= all) target = all - 1;
    const uint32_t tile = (uint32_t)__builtin_ctzll(__ballot(tile_upto > target));
    target -= of_lane(tile_upto - tile_mass, tile);
    __syncthreads();
    const uint32_t first = tile * a.tile_segs, segs = a.segs - first < a.tile_segs ? a.segs - first : a.tile_segs;      // at most 64
    constexpr uint32_t AHEAD = 4;
    {
        Eight<T> e[AHEAD];
#pragma unroll
        for (uint32_t i = 0; i < AHEAD; ++i) e[i].load(z, first + (wave + i * WAVES < segs ? wave + i * WAVES : 0), vocab);
#pragma unroll
        for (uint32_t i = 0; i < AHEAD; ++i) {
            if (wave + i * WAVES >= segs) break;
            float v[8];
            e[i].values(v, first + wave + i * WAVES, vocab);
            uint64_t sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += drawn(v[j], e[i].first + j);
            sum = wave_sum(sum);
            if (lane == 0) s.seg_sum[wave + i * WAVES] = sum;
        }
    }
    __syncthreads();
    if (wave == 0) {
        const uint64_t mine = lane < segs ? s.seg_sum[lane] : 0, upto = wave_scan(mine);
        const uint32_t seg = (uint32_t)__builtin_ctzll(__ballot(upto > target));
        pick_in_segment(a, r, row, z, first + seg, target - of_lane(upto - mine, seg), (double)top, __builtin_ldexp((double)all, -a.bits), drawn);
    }
    return true;
}

// Selections over the whole row: any number of equal logits, infinite ones, any vocabulary.
template <typename T>
__device__ __forceinline__ void pick_slow(const SampleArgs& a, const Rules& r, int64_t row, Lds& s) {
    const int64_t vocab = a.vocab;
    const T* z = (const T*)a.z + row * a.z_stride;
    const uint32_t tid = threadIdx.x;
    auto each = [&](auto f) {
#pragma unroll 1
        for (int64_t i = tid; i < vocab; i += THREADS) {
            const uint32_t key = key_of(to_f32(z[i]));
            if (key) f(key, i);
        }
    };
    uint32_t top = 0;
    uint64_t valid = 0;
    each([&](uint32_t key, int64_t) {
        top = larger(top, key);
        ++valid;
    });
    top = wave_max(top);
    __syncthreads();
    if ((tid & 63) == 0) s.words[tid >> 6] = top;
    __syncthreads();
    top = wave_max(s.words[tid & (WAVES - 1)]);
    valid = block_sum(valid, s);
    if (top == 0) {
        if (tid == 0) {
            a.token[row] = -1;
            if (a.logprob) a.logprob[row] = -__builtin_inff();
        }
        return;
    }
    const bool infinite = top == KEY_INF;
    const Weigh w{(double)logit_of(top), r.per_logit, s.table};
    auto units = [&](uint32_t key) -> uint64_t { return infinite ? (uint64_t)(key == top) << a.bits : w.units(logit_of(key), a.bits); };
    const int64_t k = r.greedy ? 1 : r.k;
    uint32_t floor = 0;
    uint64_t ties = ~0ull, before;
    if (k && (uint64_t)k < valid) {
        floor = select(s, (uint64_t)k, before, [&](auto add) { each([&](uint32_t key, int64_t) { add(key, 1); }); });
        ties = (uint64_t)k - before;
    }
    if (r.p < 1.0f && !r.greedy) {
        uint64_t sum = 0;
        each([&](uint32_t key, int64_t) { if (key > floor) sum += units(key); });
        sum = block_sum(sum, s) + (floor ? ties * units(floor) : 0);
        uint64_t want = (uint64_t)ceil(fmax(r.p, 0.0f) * (double)sum);
        if (want < 1) want = 1;
        const uint32_t key = select(s, want, before, [&](auto add) {
            each([&](uint32_t key, int64_t) { if (key > floor) add(key, units(key)); });
            if (floor && tid == 0) add(floor, ties * units(floor));
        });
        const uint64_t unit = units(key);
        const uint64_t n = unit ? (want - before + unit - 1) / unit : ~0ull;
        if (key == floor) ties = n < ties ? n : ties;
        else {
            floor = key;
            ties = n;
        }
    }
    int64_t limit = vocab;
    if (floor) {
        uint64_t n = 0;
        each([&](uint32_t key, int64_t) { n += key == floor; });
        n = block_sum(n, s);
        if (ties < n)
            limit = ~select(s, ties, before, [&](auto add) { each([&](uint32_t key, int64_t i) { if (key == floor) add(~(uint32_t)i, 1); }); });
    }
    auto drawn = [&](uint32_t key, int64_t i) -> uint64_t {
        if (key < floor || (key == floor && i > limit)) return 0;
        if (!r.greedy && r.least > 0.0f && !infinite && !(w.real(logit_of(key)) >= (double)r.least)) return 0;
        return r.greedy ? 1 : units(key);
    };
    uint64_t total = 0;
    each([&](uint32_t key, int64_t i) { total += drawn(key, i); });
    total = block_sum(total, s);
    float uf = a.u[row];
    if (!(uf > 0.0f)) uf = 0.0f;
    uint64_t target = (uint64_t)((double)uf * (double)total);
    if (target >= total) target = total - 1;
    uint64_t done = 0;
#pragma unroll 1
    for (int64_t from = 0; from < vocab; from += THREADS) {
        const int64_t i = from + tid;
        const uint32_t key = i < vocab ? key_of(to_f32(z[i])) : 0u;
        const uint64_t d = key ? drawn(key, i) : 0;
        uint64_t all;
        const uint64_t at = done + block_scan(d, s, all);
        if (d && at <= target && target < at + d) {
            a.token[row] = (int32_t)i;
            const double x = infinite ? 0.0 : ((double)logit_of(key) - (double)logit_of(top)) * r.per_nat;
            if (a.logprob) a.logprob[row] = r.greedy ? 0.0f : (float)(x - log(__builtin_ldexp((double)total, -a.bits)));
        }
        done += all;
        if (done > target) break;
    }
}

template <typename T>
__global__ __launch_bounds__(THREADS) void k_pick(SampleArgs a) {
    __shared__ Lds s;
    const int64_t row = blockIdx.x;
    const Rules r = rules_of(a, row);
    fill_table(s.table);
    __syncthreads();
    if (a.segs > MAX_SEGS || !pick_fast<T>(a, r, row, s)) pick_slow<T>(a, r, row, s);
}

// How a call's work is laid out.
struct Plan {
    int64_t segs, tiles, tile_segs;
    int64_t top_bytes, seg_bytes, bin_bytes, count_bytes, bytes;
};
Plan plan_for(int64_t rows, int64_t vocab) {
    Plan p{};
    p.segs = (vocab + SEG - 1) / SEG;
    if (p.segs > MAX_SEGS || p.segs == 0) return p;
    p.tile_segs = (p.segs + 15) / 16;             // 16 tiles of up to 64 segments
    p.tiles = (p.segs + p.tile_segs - 1) / p.tile_segs;
    auto round = [](int64_t n) { return (n + 15) / 16 * 16; };
    p.top_bytes = round(rows * p.segs * 4);
    p.seg_bytes = round(rows * p.segs * 8);
    p.bin_bytes = rows * p.tiles * BINS * 8;
    p.count_bytes = rows * p.tiles * BINS * 4;
    p.bytes = p.top_bytes + p.seg_bytes + p.bin_bytes + p.count_bytes;
    return p;
}

template <typename T>
int launch_sample(const SampleArgs& a, int64_t rows, hipStream_t stream) {
    if (a.segs >= 1 && a.segs <= MAX_SEGS) {
        const int64_t waves = rows * a.segs;
        const int per = waves >= 16384 ? 4 : 1;
        const int64_t blocks = ((int64_t)a.segs + 4 * per - 1) / (4 * per);
        if (rows * blocks > most_blocks(256) || rows * a.tiles > most_blocks(256)) return MOEQ8_EUNSUPPORTED;
        const dim3 grid((uint32_t)(rows * blocks));
        if (per == 4) hipLaunchKernelGGL((k_scan<T, 4>), grid, dim3(256), 0, stream, a, (uint32_t)blocks);
        else hipLaunchKernelGGL((k_scan<T, 1>), grid, dim3(256), 0, stream, a, (uint32_t)blocks);
        if (a.top_k || a.top_p || a.min_p)
            hipLaunchKernelGGL((k_bins<T>), dim3((uint32_t)(rows * a.tiles)), dim3(256), 0, stream, a);
    }
    hipLaunchKernelGGL((k_pick<T>), dim3((uint32_t)rows), dim3(THREADS), 0, stream, a);
    return check_launch();
}

}  // namespace
}  // namespace moeq8

extern "C" size_t logits_sample_workspace_bytes(int64_t n_rows, int64_t vocab) {
    using namespace moeq8;
    if (n_rows < 1 || vocab < 1 || vocab >= (1 << 30) || n_rows > most_blocks(THREADS)) return 0;
    return (size_t)plan_for(n_rows, vocab).bytes;
}

extern "C" int logits_sample(const void* logits, int64_t logits_row_stride, int32_t dtype, int64_t n_rows, int64_t vocab,
                             const float* u, const float* temperature, const int32_t* top_k, const float* top_p,
                             const float* min_p, int32_t* token, float* logprob, void* workspace, size_t workspace_bytes,
                             void* stream) {
    using namespace moeq8;
    if (dtype < MOEQ8_F32 || dtype > MOEQ8_BF16 || n_rows < 0 || vocab < 0) return MOEQ8_EINVAL;
    if (n_rows > 1 && logits_row_stride < vocab) return MOEQ8_EINVAL;
    if (n_rows && ((vocab && !logits) || !u || !token)) return MOEQ8_EINVAL;
    if (vocab >= (1 << 30)) return MOEQ8_EUNSUPPORTED;
    const int es = dtype_bytes(dtype);
    if ((uintptr_t)logits & (uintptr_t)(es - 1)) return MOEQ8_EALIGN;
    if (((uintptr_t)u | (uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p | (uintptr_t)min_p | (uintptr_t)token |
         (uintptr_t)logprob) & 3u)
        return MOEQ8_EALIGN;
    if (n_rows == 0) return MOEQ8_OK;
    if (n_rows > most_blocks(THREADS)) return MOEQ8_EUNSUPPORTED;
    const Plan p = plan_for(n_rows, vocab);
    if (p.bytes && (!workspace || workspace_bytes < (size_t)p.bytes)) return MOEQ8_EINVAL;
    if (p.bytes && (uintptr_t)workspace & 15u) return MOEQ8_EALIGN;
    // what is written lies apart from itself and from what other blocks still read
    const int64_t z_bytes = ((n_rows - 1) * logits_row_stride + vocab) * es, n_bytes = 4 * n_rows;
    const struct { const void* p; int64_t bytes; } all[] = {
        {workspace, p.bytes}, {token, n_bytes}, {logprob, n_bytes}, {logits, z_bytes}, {u, n_bytes},
        {temperature, n_bytes}, {top_k, n_bytes}, {top_p, n_bytes}, {min_p, n_bytes}};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 9; ++j)
            if (all[i].p && all[j].p && all[i].bytes && ranges_overlap(all[i].p, all[i].bytes, all[j].p, all[j].bytes))
                return MOEQ8_EINVAL;
    int bits = 51;
    while (vocab > (1ll << (63 - bits))) --bits;
    uint8_t* ws = (uint8_t*)workspace;
    const SampleArgs a{logits, logits_row_stride, vocab, u, temperature, top_p, min_p, top_k, token, logprob, bits,
                       (uint32_t)p.segs, (uint32_t)p.tiles, (uint32_t)p.tile_segs, (uint32_t*)ws,
                       (uint64_t*)(ws + p.top_bytes), (uint64_t*)(ws + p.top_bytes + p.seg_bytes),
                       (uint32_t*)(ws + p.top_bytes + p.seg_bytes + p.bin_bytes)};
    switch (dtype) {
        case MOEQ8_F32: return launch_sample<float>(a, n_rows, (hipStream_t)stream);
        case MOEQ8_F16: return launch_sample<f16_t>(a, n_rows, (hipStream_t)stream);
        default: return launch_sample<bf16_t>(a, n_rows, (hipStream_t)stream);
    }
}
