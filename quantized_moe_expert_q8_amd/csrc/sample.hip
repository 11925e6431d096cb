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
// largest passes it; else the bin that the threshold falls into.  The draw takes the
// segment first, then its logits in order.  Rows with more candidates than LDS holds
// (equal logits by the thousand), with infinite logits, or of over 524288 logits go
// the slow way: selections over the whole row.
#include "moeq8_cache.hpp"
#include "moeq8_lds.hpp"

namespace moeq8 {
namespace {

constexpr int SEG = 512;                          // logits a segment: 8 a lane
constexpr int MAX_SEGS = 1024;                    // more: the slow way
constexpr int BINS = 1024, PER_OCTAVE = 64;       // steps of the exponent's table; a bin is 4 of them
constexpr int CAP = 6144;                         // candidates that k_pick holds
constexpr int THREADS = 1024, WAVES = THREADS / 64;
constexpr int FEW_HITS = 96;                      // segments that pass min-p: candidates at once

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
constexpr uint32_t KEY_INF = 0xff800000u;

// A row's rules.
struct Rules {
    int64_t k;                                    // 0: all
    float p, least;                               // 1 and 0: all
    bool greedy;
    double per_logit;                             // steps of the exponent's table a logit: 64 log2(e) / T
    double per_nat;                               // 1 / T
    __device__ bool pure() const { return !greedy && !k && p == 1.0f && least == 0.0f; }
    // whether k_scan sums the masses: for the draw, or for top-p beside min-p
    __device__ bool masses() const { return !greedy && !k && (p < 1.0f) == (least > 0.0f); }
};
__device__ Rules rules_of(const SampleArgs& a, int64_t row) {
    Rules r;
    const float t = a.temperature ? a.temperature[row] : 1.0f;
    r.greedy = !(t > 0.0f);
    r.k = a.top_k ? a.top_k[row] : 0;
    if (r.k < 0 || r.k >= a.vocab) r.k = 0;
    r.p = a.top_p ? a.top_p[row] : 1.0f;
    if (!(r.p < 1.0f)) r.p = 1.0f;
    r.least = a.min_p ? a.min_p[row] : 0.0f;
    if (!(r.least > 0.0f)) r.least = 0.0f;
    if (r.least > 1.0f) r.least = 1.0f;
    r.per_nat = 1.0 / (double)t;
    r.per_logit = (PER_OCTAVE * 1.4426950408889634) / (double)t;
    return r;
}

// Weights below a largest logit.  2^(t / 64) with t = i + r, i the nearest integer:
// 2^((i mod 64) / 64) from a table, 2^(r / 64) by its Taylor series, whose sixth term
// is below 2^-54.
struct Weigh {
    double top, c;                                // the largest logit; table steps a logit
    const double* table;                          // 2^(j / 64)
    __device__ __forceinline__ double steps(float z) const { return fmax(((double)z - top) * c, -64.0 * PER_OCTAVE); }
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
    __device__ __forceinline__ uint64_t units(float z, int bits, int& i) const {
        const double v = __builtin_ldexp(at(steps(z), i), (i >> 6) + bits) + 0x1p52;
        return __builtin_bit_cast(uint64_t, v) & ((1ull << 52) - 1);
    }
    __device__ __forceinline__ uint64_t units(float z, int bits) const {
        int i;
        return units(z, bits, i);
    }
};
__device__ __forceinline__ int bin_of(int i) {    // i <= 0
    const int b = -i >> 2;
    return b < BINS ? b : BINS - 1;
}
__device__ __forceinline__ int bin_of(const Weigh& w, float z) { return bin_of((int)rint(w.steps(z))); }

__device__ __forceinline__ void fill_table(double* table) {
    if (threadIdx.x < PER_OCTAVE) table[threadIdx.x] = exp2((double)threadIdx.x / PER_OCTAVE);
}

// Eight logits of a segment from element `at` on; NaN past the row.
template <typename T>
__device__ __forceinline__ void load8(float (&v)[8], const T* z, int64_t at, int64_t vocab) {
    if (at + 8 <= vocab) {
        T raw[8];
        load_vec(raw, z + at);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = to_f32(raw[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = at + j < vocab ? to_f32(z[at + j]) : __builtin_nanf("");
    }
}

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
// Sum over the lanes up to this one.
template <typename V>
__device__ __forceinline__ V wave_scan(V v) {
    for (int i = 1; i < 64; i <<= 1) {
        const V t = __shfl_up(v, i);
        if ((int)(threadIdx.x & 63) >= i) v += t;
    }
    return v;
}

// ---- segments --------------------------------------------------------------------

template <typename T, int PER>
__global__ __launch_bounds__(256) void k_scan(SampleArgs a, uint32_t blocks) {
    __shared__ double table[PER_OCTAVE];
    const uint32_t row = blockIdx.x / blocks, block = blockIdx.x - row * blocks;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const T* z = (const T*)a.z + row * a.z_stride;
    const uint32_t first = (block * 4 + wave) * PER;
    float v[PER][8];
#pragma unroll
    for (int s = 0; s < PER; ++s) load8(v[s], z, (int64_t)(first + s) * SEG + lane * 8, a.vocab);
    const Rules r = rules_of(a, row);
    const bool masses = r.masses();
    if (masses) {
        fill_table(table);
        __syncthreads();
    }
#pragma unroll
    for (int s = 0; s < PER; ++s) {
        if (first + s >= a.segs) break;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = larger(top, key_of(v[s][j]));
        top = wave_max(top);
        uint64_t sum = 0;
        if (masses && top) {
            const Weigh w{(double)logit_of(top), r.per_logit, table};
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += v[s][j] > -__builtin_inff() ? w.units(v[s][j], 51) : 0;
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
    uint32_t key;                                 // largest key of this thread's segment
    uint32_t top;                                 // of the row
    Way way;
};

// Needs 2 * WAVES dwords of LDS; every thread of the block calls it.
__device__ Row row_of(const SampleArgs& a, const Rules& r, int64_t row, uint32_t* lds, const double* table) {
    Row o;
    const uint32_t tid = threadIdx.x;
    o.key = tid < a.segs ? a.seg_top[row * a.segs + tid] : 0u;
    const uint32_t most = wave_max(o.key);
    if ((tid & 63) == 0) lds[tid >> 6] = most;
    __syncthreads();
    o.top = 0;
    for (int i = 0; i < WAVES; ++i) o.top = larger(o.top, lds[i]);
    // segments with a logit to draw, and those that pass min-p
    const Weigh w{(double)logit_of(o.top), r.per_logit, table};
    const bool some = o.key != 0, passes = some && o.top != KEY_INF && w.real(logit_of(o.key)) >= (double)r.least;
    const uint32_t packed = (uint32_t)__popcll(__ballot(some)) | (uint32_t)__popcll(__ballot(passes)) << 16;
    if ((tid & 63) == 0) lds[WAVES + (tid >> 6)] = packed;
    __syncthreads();
    uint32_t counts = 0;
    for (int i = 0; i < WAVES; ++i) counts += lds[WAVES + i];
    const uint32_t segs = counts & 0xffffu, hits = counts >> 16;
    if (o.top == 0) o.way = NONE;
    else if (r.greedy) o.way = GREEDY;
    else if (o.top == KEY_INF) o.way = SLOW;
    else if (r.pure()) o.way = PURE;
    else if (segs <= CAP / SEG) o.way = LIST;
    else if (r.k) o.way = r.k <= segs * 3 / 4 ? LIST : BY_BINS;
    else if (r.least > 0.0f && hits <= FEW_HITS) o.way = LIST;
    else o.way = BY_BINS;
    return o;
}

// ---- bins --------------------------------------------------------------------------

template <typename T>
__global__ __launch_bounds__(THREADS) void k_bins(SampleArgs a) {
    __shared__ double table[PER_OCTAVE];
    __shared__ uint32_t words[2 * WAVES];
    __shared__ unsigned long long mass[BINS];
    __shared__ uint32_t count[BINS];
    const uint32_t row = blockIdx.x / a.tiles, tile = blockIdx.x - row * a.tiles, tid = threadIdx.x;
    const Rules r = rules_of(a, row);
    if (r.greedy || (!r.k && r.p == 1.0f)) return;        // min-p alone needs no bins
    fill_table(table);
    mass[tid] = 0;
    count[tid] = 0;
    __syncthreads();
    const Row o = row_of(a, r, row, words, table);
    if (o.way != BY_BINS) return;
    const Weigh w{(double)logit_of(o.top), r.per_logit, table};
    const T* z = (const T*)a.z + row * a.z_stride;
    const uint32_t first = tile * a.tile_segs, last = first + a.tile_segs < a.segs ? first + a.tile_segs : a.segs;
    for (int64_t at = (int64_t)first * SEG + tid * 8; at < (int64_t)last * SEG; at += THREADS * 8) {
        float v[8];
        load8(v, z, at, a.vocab);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (!(v[j] > -__builtin_inff())) continue;
            int i;
            const uint64_t u = w.units(v[j], a.bits, i);
            const int b = bin_of(i);
            atomicAdd(&mass[b], (unsigned long long)u);
            if (r.k) atomicAdd(&count[b], 1u);
        }
    }
    __syncthreads();
    const int64_t at = ((int64_t)row * a.tiles + tile) * BINS + tid;
    a.bin_mass[at] = mass[tid];
    if (r.k) a.bin_count[at] = count[tid];
}

// ---- the pick ------------------------------------------------------------------------

struct Lds {
    double table[PER_OCTAVE];
    uint64_t seg_sum[MAX_SEGS];
    uint64_t hist[256];
    uint64_t sums[WAVES];
    uint64_t pick_before;
    uint32_t words[2 * WAVES];
    uint32_t pick_key, n, seg;
    uint64_t rest;
    uint16_t hit[MAX_SEGS];
    uint32_t key[CAP], index[CAP];
};

// Sum over the block; every thread gets it.
__device__ uint64_t block_sum(uint64_t v, Lds& s) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s.sums[threadIdx.x >> 6] = v;
    __syncthreads();
    uint64_t t = 0;
    for (int i = 0; i < WAVES; ++i) t += s.sums[i];
    return t;
}
// Sum over the threads before this one, and over all.
template <typename V>
__device__ V block_scan(V v, Lds& s, V& all) {
    const V up_to = wave_scan(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 63) s.sums[threadIdx.x >> 6] = __builtin_bit_cast(uint64_t, up_to);
    __syncthreads();
    V before = 0;
    all = 0;
    for (int i = 0; i < WAVES; ++i) {
        const V t = __builtin_bit_cast(V, s.sums[i]);
        if (i < (int)(threadIdx.x >> 6)) before += t;
        all += t;
    }
    return before + up_to - v;
}

// The key from which on, in falling order, the sum reaches `want` (or the last one),
// and the sum before it.  each(f) calls f(key, amount) for this thread's part.
template <typename E>
__device__ uint32_t select(Lds& s, uint64_t want, uint64_t& before, E each) {
    uint32_t prefix = 0;
    before = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        __syncthreads();
        if (threadIdx.x < 256) s.hist[threadIdx.x] = 0;
        __syncthreads();
        each([&](uint32_t key, uint64_t amount) {
            if (shift == 24 || (key ^ prefix) >> (shift + 8) == 0)
                atomicAdd((unsigned long long*)&s.hist[key >> shift & 255], (unsigned long long)amount);
        });
        __syncthreads();
        if (threadIdx.x < 64) {                   // lane l has the four digits from 255 - 4 l down
            uint64_t h[4], sum = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += h[j] = s.hist[255 - 4 * threadIdx.x - j];
            uint64_t at = before + wave_scan((unsigned long long)sum) - sum;
            const uint64_t reach = __ballot(at + sum >= want);
            if (threadIdx.x == (reach ? (uint32_t)__builtin_ctzll(reach) : 63u)) {
                int j = 0;
                while (j < 3 && at + h[j] < want) at += h[j++];
                s.pick_key = prefix | (255 - 4 * threadIdx.x - j) << shift;
                s.pick_before = at;
            }
        }
        __syncthreads();
        prefix = s.pick_key;
        before = s.pick_before;
    }
    return prefix;
}

template <typename T>
__device__ void pick_slow(const SampleArgs& a, const Rules& r, int64_t row, Lds& s);

template <typename T>
__global__ __launch_bounds__(THREADS) void k_pick(SampleArgs a) {
    __shared__ Lds s;
    const int64_t row = blockIdx.x;
    const T* z = (const T*)a.z + row * a.z_stride;
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Rules r = rules_of(a, row);
    fill_table(s.table);
    __syncthreads();
    if (a.segs > MAX_SEGS) {
        pick_slow<T>(a, r, row, s);
        return;
    }
    const Row o = row_of(a, r, row, s.words, s.table);
    if (o.way == NONE) {
        if (tid == 0) {
            a.token[row] = -1;
            if (a.logprob) a.logprob[row] = -__builtin_inff();
        }
        return;
    }
    if (o.way == SLOW) {
        pick_slow<T>(a, r, row, s);
        return;
    }
    const float top = logit_of(o.top);
    const Weigh w{(double)top, r.per_logit, s.table};

    // ---- greedy: the first of the largest ----
    if (o.way == GREEDY) {
        if (tid == 0) s.seg = ~0u;
        __syncthreads();
        if (o.key == o.top) atomicMin(&s.seg, tid);
        __syncthreads();
        if (wave == 0) {
            float v[8];
            load8(v, z, (int64_t)s.seg * SEG + lane * 8, a.vocab);
            uint32_t at = ~0u;
#pragma unroll
            for (int j = 7; j >= 0; --j)
                if (key_of(v[j]) == o.top) at = lane * 8 + j;
            const uint64_t has = __ballot(at != ~0u);
            if (lane == (uint32_t)__builtin_ctzll(has)) {
                a.token[row] = (int32_t)(s.seg * SEG + at);
                if (a.logprob) a.logprob[row] = 0.0f;
            }
        }
        return;
    }

    float uf = a.u[row];
    if (!(uf > 0.0f)) uf = 0.0f;

    // thresholds: kept are, of the keys from `from` on, those above `floor` and those
    // equal to it up to index `limit`, and of these the ones that pass min-p
    uint32_t floor = 0, from = 1;
    int64_t limit = a.vocab;
    auto kept = [&](float v, int64_t i) {
        const uint32_t key = key_of(v);
        return key >= from && (key > floor || (key == floor && i <= limit));
    };
    // weight of a logit in the draw
    auto drawn = [&](float v, int64_t i) -> uint64_t {
        if (!kept(v, i)) return 0;
        if (r.least > 0.0f && !(w.real(v) >= (double)r.least)) return 0;
        return w.units(v, a.bits);
    };
    // the mass that is drawn from, in units of the largest weight
    double mass = 0.0;

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
        mass = all;
    } else {
        // ---- candidates ----
        const bool by_bins = o.way == BY_BINS;
        uint64_t bin_mass = 0;                    // of bin `tid`
        uint32_t bin_count = 0;
        if (by_bins && (r.k || r.p < 1.0f)) {
            for (uint32_t t = 0; t < a.tiles; ++t) {
                bin_mass += a.bin_mass[(row * a.tiles + t) * BINS + tid];
                if (r.k) bin_count += a.bin_count[(row * a.tiles + t) * BINS + tid];
            }
        }
        uint32_t held_bin = ~0u;                  // the bin whose logits are in the list

        // the candidates: logits that pass(value, key) in the segments with use(largest key)
        auto gather = [&](auto use, auto pass) {
            if (tid == 0) s.n = 0;
            const bool hit = o.key && use(o.key);
            uint64_t all;
            const uint64_t at = block_scan((uint64_t)hit, s, all);
            if (hit) s.hit[at] = (uint16_t)tid;
            __syncthreads();
            constexpr int AHEAD = 4;
            for (uint32_t h = wave; h < all; h += WAVES * AHEAD) {
                float v[AHEAD][8];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const uint32_t e = h + i * WAVES < all ? h + i * WAVES : h;
                    load8(v[i], z, (int64_t)s.hit[e] * SEG + lane * 8, a.vocab);
                }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    if (h + i * WAVES >= all) break;
                    const uint32_t base = s.hit[h + i * WAVES] * SEG + lane * 8;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t key = key_of(v[i][j]);
                        if (key && pass(v[i][j], key)) {
                            const uint32_t e = atomicAdd(&s.n, 1u);
                            if (e < CAP) {
                                s.key[e] = key;
                                s.index[e] = base + j;
                            }
                        }
                    }
                }
            }
            __syncthreads();
            return s.n <= CAP;
        };
        auto listed = [&](auto f) {
            for (uint32_t e = tid; e < s.n; e += THREADS) f(s.key[e], s.index[e]);
        };

        // the first bin up to which there are `want`, and what lies before it
        auto bin_reaching = [&](uint64_t amount, uint64_t want, uint64_t& before) {
            uint64_t all;
            const uint64_t at = block_scan(amount, s, all);
            __syncthreads();
            if (tid == 0) s.seg = BINS - 1;
            __syncthreads();
            if (at < want && at + amount >= want) {
                s.seg = tid;
                s.rest = at;
            }
            __syncthreads();
            before = s.rest;
            return s.seg;
        };

        uint64_t ties = ~0ull;                    // of those equal to the threshold
        uint64_t z_mass = 0;                      // what top-p is a part of
        bool whole = false;                       // every logit above the threshold is in the list
        if (!by_bins) {
            if (r.k && r.k <= (int64_t)a.segs) {
                uint64_t before;
                from = select(s, (uint64_t)r.k, before, [&](auto add) { if (o.key) add(o.key, 1); });
                // fewer segments than k have a logit: all of their logits
                uint64_t all;
                block_scan((uint64_t)(o.key != 0), s, all);
                if (all < (uint64_t)r.k) from = 1;
            }
            const bool by_least = !r.k && r.least > 0.0f;
            const bool fits = gather([&](uint32_t key) { return key >= from && (!by_least || w.real(logit_of(key)) >= (double)r.least); },
                                     [&](float v, uint32_t key) { return key >= from && (!by_least || w.real(v) >= (double)r.least); });
            if (!fits) {
                pick_slow<T>(a, r, row, s);
                return;
            }
            whole = true;
            if (r.k && (uint64_t)r.k < s.n) {
                uint64_t before;
                floor = select(s, (uint64_t)r.k, before, [&](auto add) { listed([&](uint32_t key, uint32_t) { add(key, 1); }); });
                ties = (uint64_t)r.k - before;
            }
            if (r.p < 1.0f) {
                if (by_least) {                   // of all logits, not of the list
                    double all;
                    block_scan(o.key ? (double)a.seg_mass[row * a.segs + tid] * 0x1p-51 * w.real(logit_of(o.key)) : 0.0, s, all);
                    z_mass = (uint64_t)rint(__builtin_ldexp(all, a.bits));
                } else {
                    uint64_t sum = 0;
                    listed([&](uint32_t key, uint32_t) { if (key > floor) sum += w.units(logit_of(key), a.bits); });
                    z_mass = block_sum(sum, s) + (floor ? ties * w.units(logit_of(floor), a.bits) : 0);
                }
            }
        } else {
            // the logits of one bin; false if they are too many
            auto hold = [&](uint32_t bin) {
                held_bin = bin;
                return gather([&](uint32_t key) { return bin_of(w, logit_of(key)) <= (int)bin; },
                              [&](float v, uint32_t) { return bin_of(w, v) == (int)bin; });
            };
            uint64_t above = 0;                   // mass above the held bin
            if (r.k) {
                uint64_t all, before;
                block_scan((uint64_t)bin_count, s, all);
                if ((uint64_t)r.k < all) {
                    const uint32_t bin = bin_reaching(bin_count, (uint64_t)r.k, before);
                    if (!hold(bin)) {
                        pick_slow<T>(a, r, row, s);
                        return;
                    }
                    uint64_t in_bin;
                    floor = select(s, (uint64_t)r.k - before, in_bin, [&](auto add) { listed([&](uint32_t key, uint32_t) { add(key, 1); }); });
                    ties = (uint64_t)r.k - before - in_bin;
                    // the bins' masses without what top-k drops
                    uint64_t sum = 0;
                    listed([&](uint32_t key, uint32_t) { if (key > floor) sum += w.units(logit_of(key), a.bits); });
                    sum = block_sum(sum, s) + ties * w.units(logit_of(floor), a.bits);
                    bin_mass = tid < bin ? bin_mass : (tid == bin ? sum : 0);
                }
            }
            if (r.p < 1.0f) {
                block_scan(bin_mass, s, z_mass);
                uint64_t want = (uint64_t)ceil(fmax(r.p, 0.0f) * (double)z_mass);
                if (want < 1) want = 1;
                const uint32_t bin = bin_reaching(bin_mass, want, above);
                if (bin != held_bin && !hold(bin)) {
                    pick_slow<T>(a, r, row, s);
                    return;
                }
                // (top-k's threshold and ties, if in this bin, count as in the list's case)
                uint64_t in_bin;
                const uint32_t k_floor = floor;
                const uint64_t k_ties = ties;
                const uint64_t floor_units = k_floor ? w.units(logit_of(k_floor), a.bits) : 0;
                const bool floor_here = k_floor && bin_of(w, logit_of(k_floor)) == (int)bin;
                const uint32_t key = select(s, want - above, in_bin, [&](auto add) {
                    listed([&](uint32_t key, uint32_t) { if (key > k_floor) add(key, w.units(logit_of(key), a.bits)); });
                    if (floor_here && tid == 0) add(k_floor, k_ties * floor_units);
                });
                const uint64_t unit = w.units(logit_of(key), a.bits);
                const uint64_t n = unit ? (want - above - in_bin + unit - 1) / unit : ~0ull;
                if (key == floor) ties = n < ties ? n : ties;
                else {
                    floor = key;
                    ties = n;
                }
            }
        }
        if (!by_bins && r.p < 1.0f) {
            uint64_t want = (uint64_t)ceil(fmax(r.p, 0.0f) * (double)z_mass), sum = 0;
            if (want < 1) want = 1;
            listed([&](uint32_t key, uint32_t) { if (key > floor) sum += w.units(logit_of(key), a.bits); });
            const uint64_t floor_units = floor ? w.units(logit_of(floor), a.bits) : 0;
            sum = block_sum(sum, s) + (floor ? ties * floor_units : 0);
            if (sum >= want) {                    // else min-p cuts above top-p
                uint64_t before;
                const uint32_t key = select(s, want, before, [&](auto add) {
                    listed([&](uint32_t key, uint32_t) { if (key > floor) add(key, w.units(logit_of(key), a.bits)); });
                    if (floor && tid == 0) add(floor, ties * floor_units);
                });
                const uint64_t unit = w.units(logit_of(key), a.bits);
                const uint64_t n = unit ? (want - before + unit - 1) / unit : ~0ull;
                if (key == floor) ties = n < ties ? n : ties;
                else {
                    floor = key;
                    ties = n;
                }
            }
        }
        // the index of the last of the ties (all keys equal to the threshold are listed)
        if (floor) {
            uint64_t n = 0;
            listed([&](uint32_t key, uint32_t) { n += key == floor; });
            n = block_sum(n, s);
            if (ties < n) {
                uint64_t before;
                limit = ~select(s, ties, before, [&](auto add) { listed([&](uint32_t key, uint32_t i) { if (key == floor) add(~i, 1); }); });
            }
        }
        // ---- the kept mass by segments ----
        __syncthreads();
        s.seg_sum[tid] = 0;
        __syncthreads();
        if (whole) {
            listed([&](uint32_t key, uint32_t i) {
                const uint64_t d = drawn(logit_of(key), i);
                if (d) atomicAdd((unsigned long long*)&s.seg_sum[i / SEG], (unsigned long long)d);
            });
        } else {
            constexpr int AHEAD = 4;
            for (uint32_t h = wave; h < a.segs; h += WAVES * AHEAD) {
                float v[AHEAD][8];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    if (h + i * WAVES < a.segs) load8(v[i], z, (int64_t)(h + i * WAVES) * SEG + lane * 8, a.vocab);
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    if (h + i * WAVES >= a.segs) break;
                    uint64_t sum = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum += drawn(v[i][j], (int64_t)(h + i * WAVES) * SEG + lane * 8 + j);
                    sum = wave_sum(sum);
                    if (lane == 0) s.seg_sum[h + i * WAVES] = sum;
                }
            }
        }
        __syncthreads();
        const uint64_t mine = s.seg_sum[tid];
        uint64_t all;
        const uint64_t before = block_scan(mine, s, all);
        uint64_t target = (uint64_t)((double)uf * (double)all);
        if (target >= all) target = all - 1;
        if (mine && before <= target && target < before + mine) {
            s.seg = tid;
            s.rest = target - before;
        }
        mass = __builtin_ldexp((double)all, -a.bits);
    }
    __syncthreads();

    // ---- the token of the segment, in order: the first up to which there is more than the rest ----
    if (wave == 0) {
        const uint32_t seg = s.seg;
        const int64_t base = (int64_t)seg * SEG + lane * 8;
        float v[8];
        load8(v, z, base, a.vocab);
        const Weigh own{o.way == PURE ? (double)logit_of(s.pick_key) : w.top, w.c, s.table};
        uint64_t u[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (o.way == PURE) u[j] = v[j] > -__builtin_inff() ? own.units(v[j], 51) : 0;
            else u[j] = drawn(v[j], base + j);
            sum += u[j];
        }
        uint64_t at = wave_scan((unsigned long long)sum) - sum;
        const uint64_t past = __ballot(at + sum > s.rest), any = __ballot(sum > 0);
        const uint32_t has = past ? (uint32_t)__builtin_ctzll(past) : 63u - (uint32_t)__builtin_clzll(any);
        if (lane == has) {
            int pick = 0;
            for (int j = 0; j < 8; ++j) {
                if (u[j]) pick = j;
                at += u[j];
                if (u[j] && at > s.rest) break;
            }
            a.token[row] = (int32_t)(base + pick);
            if (a.logprob) a.logprob[row] = (float)(((double)v[pick] - (double)top) * r.per_nat - log(mass));
        }
    }
}

// Selections over the whole row: any number of equal logits, infinite ones, any vocabulary.
template <typename T>
__device__ __attribute__((noinline)) void pick_slow(const SampleArgs& a, const Rules& r, int64_t row, Lds& s) {
    const int64_t vocab = a.vocab;
    const T* z = (const T*)a.z + row * a.z_stride;
    const uint32_t tid = threadIdx.x;
    auto each = [&](auto f) {
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
    for (int i = 0; i < WAVES; ++i) top = larger(top, s.words[i]);
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

// How a call's work is laid out.
struct Plan {
    int64_t segs, tiles, tile_segs;
    int64_t top_bytes, seg_bytes, bin_bytes, count_bytes, bytes;
};
Plan plan_for(int64_t rows, int64_t vocab) {
    Plan p{};
    p.segs = (vocab + SEG - 1) / SEG;
    if (p.segs > MAX_SEGS || p.segs == 0) return p;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(16, 1024 / rows));
    p.tile_segs = (p.segs + want - 1) / want;
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
        if (rows * blocks > most_blocks(256) || rows * a.tiles > most_blocks(THREADS)) return MOEQ8_EUNSUPPORTED;
        const dim3 grid((uint32_t)(rows * blocks));
        if (per == 4) hipLaunchKernelGGL((k_scan<T, 4>), grid, dim3(256), 0, stream, a, (uint32_t)blocks);
        else hipLaunchKernelGGL((k_scan<T, 1>), grid, dim3(256), 0, stream, a, (uint32_t)blocks);
        if (a.top_k || a.top_p || a.min_p)
            hipLaunchKernelGGL((k_bins<T>), dim3((uint32_t)(rows * a.tiles)), dim3(THREADS), 0, stream, a);
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
