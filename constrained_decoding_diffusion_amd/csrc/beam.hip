// Beam search under the automaton: the joint selection of K hypotheses over
// beams and vocabulary, and the lookahead that keeps them out of dead ends.
//
// key(k, v) = s_k + x_k[v] - lse_k over the tokens v that an edge out of the
// hypothesis' state set holds.  Within one beam the keys order as the values
// x_k[v], so one pass over x (beam_scan) needs no selection at all: it leaves
// the log-sum-exp partials and, per granule of 512 tokens, the largest allowed
// value.  The K best candidates lie in the K granules with the largest maxima
// (order: key, then the lower token index; a candidate of any other granule
// has K granule maxima before it), so the second kernel (beam_pick) ranks
// the granules, reads those K again and ranks their tokens.
#include <algorithm>

#include "device_common.h"

namespace fa {
namespace {

constexpr int kScanWaves = 4;
constexpr int kMaskWords = kBeamGran / 32;
constexpr int kPickThreads = 1024;
constexpr int kPickWaves = kPickThreads / kWave;

__device__ inline bool has_bit(const uint32_t *set, int s) { return (set[s >> 5] >> (s & 31)) & 1u; }

__device__ inline float to_float(float x) { return x; }
__device__ inline float to_float(_Float16 x) { return (float)x; }
struct Bf16 {
    uint16_t u;
};
__device__ inline float to_float(Bf16 x) { return __uint_as_float((uint32_t)x.u << 16); }

// tokens v .. v+7 of a row of V; -inf past its end
template <class T>
__device__ inline void load8(const T *row, int v, int V, float (&x)[8])
{
    if (v + 8 <= V) {
        T t[8];
        __builtin_memcpy(t, row + v, sizeof(t));  // any element alignment
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = to_float(t[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = v + j < V ? to_float(row[v + j]) : -INFINITY;
    }
}

// calls fn(state) for every state of the set, one after the other, the whole
// wavefront at once
template <class Fn>
__device__ inline void each_state(const uint32_t *set, int W, int lane, Fn fn)
{
    for (int w0 = 0; w0 < W; w0 += kWave) {
        const uint32_t word = w0 + lane < W ? set[w0 + lane] : 0u;
        unsigned long long nz = __ballot(word != 0u);
        while (nz) {
            const int l = __ffsll(nz) - 1;
            nz &= nz - 1;
            uint32_t bits = __builtin_amdgcn_readlane(word, l);
            while (bits) {
                fn((w0 + l) * 32 + __ffs(bits) - 1);
                bits &= bits - 1;
            }
        }
    }
}

// mask[0 .. ng*16): bit t set when token g0*512 + t may follow the state set.
// The wavefront's own LDS words.
__device__ inline void allowed_mask(const DevTable &d, const uint32_t *set, int W,
                                    const uint32_t *reach, int g0, int ng, uint32_t *mask, int lane)
{
    const int words = ng * kMaskWords, t0 = g0 * kBeamGran, t1 = t0 + ng * kBeamGran;
    const int nG = beam_grans(d.V);
    for (int w = lane; w < words; w += kWave) mask[w] = 0u;
    wave_sync();
    each_state(set, W, lane, [&](int s) {
        const int32_t *off = d.bm_off + (size_t)s * (nG + 1);
        const int e1 = off[min(g0 + ng, nG)];
        for (int e = off[g0] + lane; e < e1; e += kWave) {
            const int tok = d.bm_ent[2 * (size_t)e], to = d.bm_ent[2 * (size_t)e + 1];
            if (!reach || has_bit(reach, to)) atomicOr(&mask[(tok - t0) >> 5], 1u << (tok & 31));
        }
        for (int i = d.bm_doff[s]; i < d.bm_doff[s + 1]; ++i) {
            const int j = d.bm_dense[2 * (size_t)i], to = d.bm_dense[2 * (size_t)i + 1];
            if (reach && !has_bit(reach, to)) continue;
            const uint32_t *bits = d.dense_bits + (size_t)j * d.dense_words;
            for (int w = lane; w < words; w += kWave) {
                const int gw = t0 / 32 + w;
                if (gw < d.dense_words) atomicOr(&mask[w], bits[gw]);
            }
        }
        // range labels: 64 segments a time, those that meet the tokens one by one
        const int s1 = d.bm_soff[s + 1];
        for (int i0 = d.bm_soff[s]; i0 < s1; i0 += kWave) {
            int lo = 0, hi = 0;
            if (i0 + lane < s1) {
                const int32_t *sg = d.bm_seg + 4 * (size_t)(i0 + lane);
                if (!reach || has_bit(reach, sg[2])) {
                    lo = max(sg[0], t0);
                    hi = min(sg[1], t1);
                }
            }
            unsigned long long hit = __ballot(lo < hi);
            while (hit) {
                const int l = __ffsll(hit) - 1;
                hit &= hit - 1;
                const int a = __builtin_amdgcn_readlane(lo, l) - t0;
                const int b = __builtin_amdgcn_readlane(hi, l) - t0;
                for (int w = (a >> 5) + lane; w <= (b - 1) >> 5; w += kWave) {
                    const uint32_t from = a > 32 * w ? ~0u << (a - 32 * w) : ~0u;
                    const uint32_t upto = b < 32 * w + 32 ? ~(~0u << (b - 32 * w)) : ~0u;
                    atomicOr(&mask[w], from & upto);
                }
            }
        }
    });
    wave_sync();
}

__device__ inline const uint32_t *set_of(const BeamSelect &a, int row, int W)
{
    return a.states_in + (size_t)row * W;
}

template <class T>
__device__ inline const T *row_of(const BeamSelect &a, int row)
{
    return static_cast<const T *>(a.logits) + (size_t)(row / a.Kin) * a.batch_stride +
           (size_t)(row % a.Kin) * a.beam_stride;
}

// 2^t for t in about [-1100, 1], to 2e-12 relative: the integer part by the
// exponent, 2^f on [-1/2, 1/2] by its degree-8 interpolation at the Chebyshev
// points.  fp64 fused multiply-adds run at the fp32 rate on this chip, and the
// library's exp spends twice the operations on its last bits.
__device__ inline double exp2_poly(double t)
{
    const double n = __builtin_rint(t);
    const double f = t - n;
    double r = 1.3255224878668817e-06;
    r = fma(r, f, 1.5310079402249296e-05);
    r = fma(r, f, 0.00015403455852453838);
    r = fma(r, f, 0.0013333450568000645);
    r = fma(r, f, 0.009618129159402558);
    r = fma(r, f, 0.05550410941205933);
    r = fma(r, f, 0.2402265069581299);
    r = fma(r, f, 0.6931471805459335);
    r = fma(r, f, 1.0);
    return __builtin_ldexp(r, (int)n);
}

// One wavefront: NG granules of one hypothesis.  The logits are asked for
// first and arrive while the mask is put together.
//
// The sum of exponentials is held in fp64 from the first term on: keys of
// different hypotheses are compared with each other, and two of them may lie
// closer than an fp32 sum over 150,000 tokens resolves.
template <class T, int MODE, int NG>
__global__ __launch_bounds__(kScanWaves *kWave) void beam_scan(DevTable d, BeamSelect a,
                                                               float *__restrict__ gmax,
                                                               double2 *__restrict__ part,
                                                               uint32_t *__restrict__ gmask, int nblk)
{
    __shared__ uint32_t sh_mask[kScanWaves][NG * kMaskWords];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row = blockIdx.x / nblk;
    const int chunk = (blockIdx.x % nblk) * kScanWaves + wave;
    const int nG = beam_grans(d.V), W = (d.S + 31) / 32;
    const int g0 = chunk * NG;
    if (g0 >= nG) return;
    if (a.status[row / a.Kin] != 0 || a.scores_in[row] == -INFINITY) return;
    const T *x = row_of<T>(a, row);
    float v[NG][8];
#pragma unroll
    for (int i = 0; i < NG; ++i) load8(x, min((g0 + i) * kBeamGran + lane * 8, d.V), d.V, v[i]);
    uint32_t *mask = sh_mask[wave];
    allowed_mask(d, set_of(a, row, W), W, a.reach, g0, NG, mask, lane);
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        const uint32_t ok = (mask[i * kMaskWords + lane / 4] >> (8 * (lane & 3))) & 255u;
        float best = -INFINITY;
        if (__ballot(ok != 0u)) {
            bool bad = false;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // the value where the bit is set, else -inf
                const int on = (int)(ok << (31 - j)) >> 31;
                const float y = __int_as_float((__float_as_int(v[i][j]) & on) | (~on & (int)0xff800000));
                best = fmaxf(best, y);
                if (MODE == FA_BEAM_PROBS) bad |= on && !(y >= 0.f && y < INFINITY);
            }
            best = wave_max_f(best);
            // a bad probability travels as a NaN maximum
            if (MODE == FA_BEAM_PROBS && __ballot(bad)) best = NAN;
            // for the second kernel, should the granule be among the best
            if (best > -INFINITY && lane < kMaskWords)
                gmask[((size_t)row * nG + g0 + i) * kMaskWords + lane] = mask[i * kMaskWords + lane];
        }
        if (lane == 0 && g0 + i < nG) gmax[(size_t)row * nG + g0 + i] = best;
        if (MODE == FA_BEAM_LOGITS) {
#pragma unroll
            for (int j = 0; j < 8; ++j) m = __builtin_elementwise_maximum(m, v[i][j]);  // a NaN stays
        }
    }
    if (MODE == FA_BEAM_LOGITS) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) m = __builtin_elementwise_maximum(m, __shfl_xor(m, o));
        double s = m;  // NaN or +inf: the row is flagged
        if (m == -INFINITY) s = 0.0;
        else if (m < INFINITY) {
            constexpr double kLog2e = 1.4426950408889634;
            s = 0.0;
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    // the difference first: it is exact, whatever the size of the logits
                    s += exp2_poly(fmax(((double)v[i][j] - (double)m) * kLog2e, -1100.0));
            s = wave_sum_d(s);
        }
        if (lane == 0) part[(size_t)row * nG + chunk] = make_double2((double)m, s);
    }
}

__device__ inline bool before(double k0, uint32_t i0, double k1, uint32_t i1)
{
    return k0 > k1 || (k0 == k1 && i0 < i1);
}

__device__ inline double wave_max_d(double x)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x = fmax(x, __shfl_xor(x, o));
    return x;
}

// The first K of the wavefront's R keys a lane (order: `before`; -inf is no
// key), written in order to out_key / out_id; returns how many.
template <int R, class Id>
__device__ inline int wave_topk(double (&key)[R], Id id_of, int K, double *out_key,
                                uint32_t *out_id, int lane)
{
    int n = 0;
    while (n < K) {
        double bk = -INFINITY;
        uint32_t bi = ~0u;
        int br = -1;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t id = id_of(r);
            if (key[r] > -INFINITY && before(key[r], id, bk, bi)) {
                bk = key[r];
                bi = id;
                br = r;
            }
        }
        const double best = wave_max_d(bk);
        if (best == -INFINITY) break;
        uint32_t low = bk == best ? bi : ~0u;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) low = min(low, (uint32_t)__shfl_xor((int)low, o));
        if (bk == best && bi == low) {
            out_key[n] = best;
            out_id[n] = low;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r == br) key[r] = -INFINITY;
        }
        ++n;
    }
    return n;
}

// ascending as x ascends; 0 for -inf (no key)
__device__ inline uint32_t ordered_key(double x)
{
    if (!(x > -INFINITY)) return 0u;
    const uint32_t u = __float_as_uint((float)x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// the largest multiple of 2^10 that at least n (<= 64) lanes' values reach
__device__ inline uint32_t nth_largest(uint32_t x, int n)
{
    uint32_t t = 0;
    for (int bit = 31; bit >= 10; --bit)
        if (__popcll(__ballot(x >= (t | (1u << bit)))) >= n) t |= 1u << bit;
    return t;
}

struct PickShared {
    double key[kPickThreads];  // candidates
    uint32_t id[kPickThreads];
    double sel_key[FA_BEAM_MAX];  // the first K of them, in order
    uint32_t sel_id[FA_BEAM_MAX];
    int cnt[kPickWaves];
    uint32_t tau[2][kPickWaves];
    int n;  // candidates found, in either round
    int n2;
};

// The candidates, unordered, in key / id: each ranked against all of them;
// those below K go to their rank in sel_key / sel_id.
__device__ inline void rank_candidates(PickShared &sh, int n, int K)
{
    if ((int)threadIdx.x < n) {
        const double mk = sh.key[threadIdx.x];
        const uint32_t mi = sh.id[threadIdx.x];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += before(sh.key[j], sh.id[j], mk, mi);
        if (rank < K) {
            sh.sel_key[rank] = mk;
            sh.sel_id[rank] = mi;
        }
    }
}

// Where more candidates tie than the list holds: the wavefronts' own first K
// one by one, and the rank of each among all wavefronts'.
template <int R, class Id>
__device__ inline int rank_by_rounds(PickShared &sh, double (&key)[R], Id id_of, int K, int lane,
                                     int wave)
{
    const int c = wave_topk(key, id_of, K, sh.key + wave * FA_BEAM_MAX, sh.id + wave * FA_BEAM_MAX, lane);
    if (lane == 0) sh.cnt[wave] = c;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < kPickWaves; ++w) total += sh.cnt[w];
    const int w0 = threadIdx.x / FA_BEAM_MAX, j0 = threadIdx.x % FA_BEAM_MAX;
    if (j0 < sh.cnt[w0]) {
        const double mk = sh.key[threadIdx.x];
        const uint32_t mi = sh.id[threadIdx.x];
        int rank = 0;
        for (int w = 0; w < kPickWaves; ++w)
            for (int j = 0; j < sh.cnt[w]; ++j)
                rank += before(sh.key[w * FA_BEAM_MAX + j], sh.id[w * FA_BEAM_MAX + j], mk, mi);
        if (rank < K) {
            sh.sel_key[rank] = mk;
            sh.sel_id[rank] = mi;
        }
    }
    __syncthreads();
    return min(total, K);
}

// appends the lanes' keys at or above the threshold to the candidate list;
// counts all of them, also those past its end
template <int R, class Take, class Id>
__device__ inline void append(PickShared &sh, int *count, const double (&key)[R], Take take, Id id_of,
                              int lane)
{
    unsigned long long hit[R];
    int c = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        hit[r] = __ballot(take(r));
        c += __popcll(hit[r]);
    }
    if (c == 0) return;
    int base = 0;
    if (lane == 0) base = atomicAdd(count, c);
    base = __builtin_amdgcn_readfirstlane(base);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if ((hit[r] >> lane) & 1ull) {
            const int at = base + __popcll(hit[r] & ((1ull << lane) - 1ull));
            if (at < kPickThreads) {
                sh.key[at] = key[r];
                sh.id[at] = id_of(r);
            }
        }
        base += __popcll(hit[r]);
    }
}

__device__ inline void load8_as(int dtype, const void *row, int v, int V, float (&x)[8])
{
    if (dtype == FA_F32) load8(static_cast<const float *>(row), v, V, x);
    else if (dtype == FA_F16) load8(static_cast<const _Float16 *>(row), v, V, x);
    else load8(static_cast<const Bf16 *>(row), v, V, x);
}

// One workgroup: one batch row.  A lane holds RG granule maxima, and eight
// tokens of RT granules a wavefront.
//
// Both rankings go by a threshold that at least K keys reach: every candidate
// at or above it is listed, and each one's rank is the number of listed ones
// before it, so no step of the work is repeated K times.  For the granules the
// threshold is the better of two that the wavefronts' lane maxima give: the
// largest of their K-th largest, and the smallest of their ceil(K/16)-th
// largest.  For the tokens it is the K-th granule maximum.
template <int MODE, int RG, int RT>
__global__ __launch_bounds__(kPickThreads) void beam_pick(DevTable d, BeamSelect a,
                                                          const float *__restrict__ gmax,
                                                          const double2 *__restrict__ part,
                                                          const uint32_t *__restrict__ gmask,
                                                          int chunks)
{
    static_assert(kPickWaves * FA_BEAM_MAX == kPickThreads, "a thread per candidate slot");
    __shared__ double sh_lse[FA_BEAM_MAX];
    __shared__ double sh_score[FA_BEAM_MAX];
    __shared__ PickShared sh;
    __shared__ int sh_bad;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nG = beam_grans(d.V), W = (d.S + 31) / 32, Kin = a.Kin, K = a.K;
    const int row0 = b * Kin, M = Kin * nG;
    const bool flagged = a.status[b] != 0;
    if (tid == 0) {
        sh_bad = 0;
        sh.n = 0;
        sh.n2 = 0;
    }
    int n = 0;
    if (!flagged) {
        float gm[RG];
#pragma unroll
        for (int r = 0; r < RG; ++r) {
            const int i = r * kPickThreads + tid;
            gm[r] = i < M ? gmax[(size_t)row0 * nG + i] : -INFINITY;
        }
        __syncthreads();
        for (int k = wave; k < Kin; k += kPickWaves) {
            const float sc = a.scores_in[row0 + k];
            double lse = MODE == FA_BEAM_LOGITS ? -INFINITY : 0.0;
            bool bad = !(sc < INFINITY);
            if (MODE == FA_BEAM_LOGITS && sc > -INFINITY && !bad) {
                double m = -INFINITY, s = 0.0;
                const double2 *pr = part + (size_t)(row0 + k) * nG;
                bool odd = false;
                for (int c = lane; c < chunks; c += kWave) {
                    m = fmax(m, pr[c].x);
                    odd |= !(pr[c].x < INFINITY);
                }
                m = wave_max_d(m);
                for (int c = lane; c < chunks; c += kWave)
                    if (pr[c].x > -INFINITY) s += pr[c].y * exp(pr[c].x - m);
                s = wave_sum_d(s);
                if (m > -INFINITY) lse = m + log(s);
                bad = __ballot(odd) != 0ull;
                if (bad) lse = -INFINITY;
            }
            if (lane == 0) {
                sh_lse[k] = lse;
                sh_score[k] = sc > -INFINITY ? (double)sc : -INFINITY;
                if (bad) atomicOr(&sh_bad, 1);
            }
        }
        __syncthreads();
        const uint32_t per_gran = nG > 1 ? 0xffffffffu / (uint32_t)nG + 1u : 0u;
        // x the value of a token or of a granule's best one
        auto key_of = [&](int k, float x) -> double {
            const double sc = sh_score[k], lse = sh_lse[k];
            if (!(x > -INFINITY) || !(sc > -INFINITY) || !(lse > -INFINITY)) return -INFINITY;
            return MODE == FA_BEAM_PROBS ? sc + log((double)x) : sc + ((double)x - lse);
        };
        int ng;
        {
            double key[RG];
            auto id_of = [&](int r) { return (uint32_t)(r * kPickThreads + tid); };
            uint32_t top = 0;
            bool bad = false;
#pragma unroll
            for (int r = 0; r < RG; ++r) {
                key[r] = -INFINITY;
                const uint32_t i = id_of(r);
                if (i < (uint32_t)M) {
                    const int k = nG > 1 ? (int)__umulhi(i, per_gran) : (int)i;
                    // a maximum of a hypothesis that was not scanned is not there
                    if (sh_score[k] > -INFINITY) {
                        bad |= MODE == FA_BEAM_PROBS && gm[r] != gm[r];
                        key[r] = key_of(k, gm[r]);
                    }
                }
                top = max(top, ordered_key(key[r]));
            }
            if (bad) atomicOr(&sh_bad, 1);
            const uint32_t most = nth_largest(top, K);
            const uint32_t some = nth_largest(top, (K + kPickWaves - 1) / kPickWaves);
            if (lane == 0) {
                sh.tau[0][wave] = most;
                sh.tau[1][wave] = some;
            }
            __syncthreads();
            uint32_t hi = 0, lo = ~0u;
            for (int w = 0; w < kPickWaves; ++w) {
                hi = max(hi, sh.tau[0][w]);
                lo = min(lo, sh.tau[1][w]);
            }
            const uint32_t tau = max(max(hi, lo), 1u);
            append(sh, &sh.n, key, [&](int r) { return ordered_key(key[r]) >= tau; }, id_of, lane);
            __syncthreads();
            ng = sh.n;
            if (ng <= kPickThreads) {
                rank_candidates(sh, ng, K);
                __syncthreads();
                ng = min(ng, K);
            } else {
                ng = rank_by_rounds(sh, key, id_of, K, lane, wave);
            }
        }
        // their tokens; none before the last of K granule maxima is lost
        const double floor_key = ng == K ? sh.sel_key[K - 1] : -INFINITY;
        {
            double key[RT * 8];
            uint32_t base[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int q = r * kPickWaves + wave;
                base[r] = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) key[r * 8 + j] = -INFINITY;
                if (q < ng) {
                    const uint32_t i = sh.sel_id[q];
                    const int k = nG > 1 ? (int)__umulhi(i, per_gran) : (int)i;
                    const int g = (int)i - k * nG, v0 = g * kBeamGran + lane * 8;
                    const uint32_t ok = (gmask[((size_t)row0 * nG + i) * kMaskWords + lane / 4] >>
                                         (8 * (lane & 3))) & 255u;
                    const size_t at = (size_t)b * a.batch_stride + (size_t)k * a.beam_stride;
                    float x[8];
                    load8_as(a.dtype, static_cast<const char *>(a.logits) + at * (a.dtype == FA_F32 ? 4 : 2),
                             min(v0, d.V), d.V, x);
                    base[r] = (uint32_t)k * (uint32_t)d.V + (uint32_t)v0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const double kk = (ok >> j) & 1u ? key_of(k, x[j]) : -INFINITY;
                        if (kk >= floor_key) key[r * 8 + j] = kk;
                    }
                }
            }
            __syncthreads();  // sel_* is read
            auto id_of = [&](int r) { return base[r / 8] + (uint32_t)(r % 8); };
            append(sh, &sh.n2, key, [&](int r) { return key[r] > -INFINITY; }, id_of, lane);
            __syncthreads();
            n = sh.n2;
            if (n <= kPickThreads) {
                rank_candidates(sh, n, K);
                __syncthreads();
                n = min(n, K);
            } else {
                n = rank_by_rounds(sh, key, id_of, K, lane, wave);
            }
        }
        const bool bad = sh_bad != 0;
        if (tid == 0) {
            const int st = bad ? FA_ROW_BADPROB : (n == 0 ? FA_ROW_INFEASIBLE : 0);
            if (st) a.status[b] = st;  // it was 0
        }
        if (bad) n = 0;
    }
    // the slots: the states of each winner's token
    for (int j = wave; j < K; j += kPickWaves) {
        const size_t o = (size_t)b * K + j;
        uint32_t *to = a.states + o * W;
        for (int w = lane; w < W; w += kWave) to[w] = 0u;
        const bool live = j < n;
        const int k = live ? (int)(sh.sel_id[j] / (uint32_t)d.V) : j % Kin;
        const int v = live ? (int)(sh.sel_id[j] % (uint32_t)d.V) : -1;
        if (lane == 0) {
            a.scores[o] = live ? (float)sh.sel_key[j] : -INFINITY;
            a.tokens[o] = v;
            a.parents[o] = k;
        }
    }
    __syncthreads();
    for (int j = wave; j < n; j += kPickWaves) {
        uint32_t *to = a.states + ((size_t)b * K + j) * W;
        const int k = (int)(sh.sel_id[j] / (uint32_t)d.V), v = (int)(sh.sel_id[j] % (uint32_t)d.V);
        each_state(set_of(a, row0 + k, W), W, lane, [&](int s) {
            auto add = [&](int t) {
                if (!a.reach || has_bit(a.reach, t)) atomicOr(&to[t >> 5], 1u << (t & 31));
            };
            const int32_t *off = d.bm_off + (size_t)s * (nG + 1) + v / kBeamGran;
            for (int e = off[0] + lane; e < off[1]; e += kWave)
                if (d.bm_ent[2 * (size_t)e] == v) add(d.bm_ent[2 * (size_t)e + 1]);
            for (int i = d.bm_doff[s] + lane; i < d.bm_doff[s + 1]; i += kWave)
                if (has_bit(d.dense_bits + (size_t)d.bm_dense[2 * (size_t)i] * d.dense_words, v))
                    add(d.bm_dense[2 * (size_t)i + 1]);
            for (int i = d.bm_soff[s] + lane; i < d.bm_soff[s + 1]; i += kWave) {
                const int32_t *sg = d.bm_seg + 4 * (size_t)i;
                if (sg[0] <= v && v < sg[1]) add(sg[2]);
            }
        });
    }
}

constexpr int kReachThreads = 1024;

// One workgroup: the states r tokens before F, from those r - 1 before it; a
// set that repeats its predecessor repeats for good.
__global__ __launch_bounds__(kReachThreads) void beam_reach(DevTable d, int L,
                                                            uint32_t *__restrict__ sets)
{
    extern __shared__ uint32_t sh_set[];  // [2][W]
    const int W = (d.S + 31) / 32, tid = threadIdx.x;
    for (int w = tid; w < 2 * W; w += kReachThreads) sh_set[w] = 0u;
    __syncthreads();
    for (int i = tid; i < d.n_acc; i += kReachThreads)
        atomicOr(&sh_set[d.acc[i] >> 5], 1u << (d.acc[i] & 31));
    __syncthreads();
    for (int w = tid; w < W; w += kReachThreads) sets[w] = sh_set[w];
    int now = 0, same = 0;
    for (int r = 1; r <= L; ++r) {
        uint32_t *cur = sh_set + now * W, *nxt = sh_set + (1 - now) * W;
        if (!same) {
            for (int q = tid; q < d.npairs; q += kReachThreads) {
                const int p = d.pair_a[q];
                if (has_bit(cur, d.pair_b[q]) && !has_bit(nxt, p)) atomicOr(&nxt[p >> 5], 1u << (p & 31));
            }
            __syncthreads();
            int diff = 0;
            for (int w = tid; w < W; w += kReachThreads) diff |= cur[w] != nxt[w];
            same = !__syncthreads_or(diff);
            for (int w = tid; w < W; w += kReachThreads) cur[w] = 0u;
            now = 1 - now;
        }
        for (int w = tid; w < W; w += kReachThreads) sets[(size_t)r * W + w] = sh_set[now * W + w];
        __syncthreads();
    }
}

__global__ __launch_bounds__(256) void beam_start(DevTable d, int64_t rows, int K,
                                                  float *__restrict__ scores,
                                                  uint32_t *__restrict__ states)
{
    const int W = (d.S + 31) / 32;
    const int64_t n = rows * K * W;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t slot = i / W;
        const int w = (int)(i % W);
        const bool first = slot % K == 0;
        states[i] = first && w == (d.start >> 5) ? 1u << (d.start & 31) : 0u;
        if (w == 0) scores[slot] = first ? 0.f : -INFINITY;
    }
}

struct ScanOut {
    float *gmax;
    double2 *part;
    uint32_t *gmask;
};

template <class T, int MODE, int NG>
int scan(const DevTable &d, const BeamSelect &a, const ScanOut &o, hipStream_t st)
{
    const int64_t waves = (beam_grans(d.V) + NG - 1) / NG;
    const int64_t nblk = (waves + kScanWaves - 1) / kScanWaves;
    const int64_t blocks = nblk * a.B * a.Kin;
    if (blocks > 0x7fffffff) return -1;
    beam_scan<T, MODE, NG><<<(unsigned)blocks, kScanWaves * kWave, 0, st>>>(d, a, o.gmax, o.part,
                                                                            o.gmask, (int)nblk);
    return (int)hipGetLastError();
}

template <int MODE, int RG, int RT>
int pick(const DevTable &d, const BeamSelect &a, const ScanOut &o, int chunks, hipStream_t st)
{
    beam_pick<MODE, RG, RT><<<a.B, kPickThreads, 0, st>>>(d, a, o.gmax, o.part, o.gmask, chunks);
    return (int)hipGetLastError();
}

template <int MODE, int RG>
int pick_tokens(const DevTable &d, const BeamSelect &a, const ScanOut &o, int chunks, hipStream_t st)
{
    if (a.K <= kPickWaves) return pick<MODE, RG, 1>(d, a, o, chunks, st);
    return pick<MODE, RG, FA_BEAM_MAX / kPickWaves>(d, a, o, chunks, st);
}

template <int MODE>
int select(const DevTable &d, const BeamSelect &a, const ScanOut &o, hipStream_t st)
{
    constexpr int NG = 4;
    const int nG = beam_grans(d.V), chunks = (nG + NG - 1) / NG;
    const int e = a.dtype == FA_F32   ? scan<float, MODE, NG>(d, a, o, st)
                  : a.dtype == FA_F16 ? scan<_Float16, MODE, NG>(d, a, o, st)
                                      : scan<Bf16, MODE, NG>(d, a, o, st);
    if (e) return e;
    if (a.Kin * nG <= 8 * kPickThreads) return pick_tokens<MODE, 8>(d, a, o, chunks, st);
    return pick_tokens<MODE, kBeamGranMax / kPickThreads>(d, a, o, chunks, st);
}

}  // namespace

BeamWs beam_ws_layout(const HostTable &t, int32_t B, int32_t Kin)
{
    auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t n = (size_t)B * Kin * beam_grans(t.V);
    BeamWs w;
    w.gmax = 0;
    w.part = al(n * sizeof(float));
    w.gmask = al(w.part + n * 2 * sizeof(double));
    w.total = al(w.gmask + n * kMaskWords * sizeof(uint32_t));
    return w;
}

int launch_beam_lookahead(const DevTable &d, int L, uint32_t *sets, void *stream)
{
    const size_t lds = 2 * (size_t)((d.S + 31) / 32) * sizeof(uint32_t);
    beam_reach<<<1, kReachThreads, lds, (hipStream_t)stream>>>(d, L, sets);
    return (int)hipGetLastError();
}

int launch_beam_start(const DevTable &d, int B, int K, float *scores, uint32_t *states, void *stream)
{
    const int64_t n = (int64_t)B * K * ((d.S + 31) / 32);
    const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, 4096);
    beam_start<<<blocks, 256, 0, (hipStream_t)stream>>>(d, B, K, scores, states);
    return (int)hipGetLastError();
}

int launch_beam_select(const DevTable &d, const BeamSelect &a, uint8_t *ws, const BeamWs &w,
                       void *stream)
{
    const ScanOut o{reinterpret_cast<float *>(ws + w.gmax), reinterpret_cast<double2 *>(ws + w.part),
                    reinterpret_cast<uint32_t *>(ws + w.gmask)};
    hipStream_t st = (hipStream_t)stream;
    return a.mode == FA_BEAM_LOGITS ? select<FA_BEAM_LOGITS>(d, a, o, st)
                                    : select<FA_BEAM_PROBS>(d, a, o, st);
}

}  // namespace fa
