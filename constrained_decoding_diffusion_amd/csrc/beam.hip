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
                                                               double2 *__restrict__ part, int nblk)
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

// rank of every wavefront's candidates among all of them; those below K go to
// their rank in out_key / out_id.  Returns how many there are (at most K).
// Ends with the workgroup in step.
__device__ inline int block_rank(const double *key, const uint32_t *id, const int *cnt, int K,
                                 double *out_key, uint32_t *out_id)
{
    __syncthreads();
    int total = 0;
    for (int w = 0; w < kPickWaves; ++w) total += cnt[w];
    const int w0 = threadIdx.x / FA_BEAM_MAX, j0 = threadIdx.x % FA_BEAM_MAX;
    if (j0 < cnt[w0]) {
        const double mk = key[threadIdx.x];
        const uint32_t mi = id[threadIdx.x];
        int rank = 0;
        for (int w = 0; w < kPickWaves; ++w)
            for (int j = 0; j < cnt[w]; ++j)
                rank += before(key[w * FA_BEAM_MAX + j], id[w * FA_BEAM_MAX + j], mk, mi);
        if (rank < K) {
            out_key[rank] = mk;
            out_id[rank] = mi;
        }
    }
    __syncthreads();
    return min(total, K);
}

// One workgroup: one batch row.  RG keys a lane hold the granules of its
// hypotheses, RT those of the K granules' tokens.
template <class T, int MODE, int RG, int RT>
__global__ __launch_bounds__(kPickThreads) void beam_pick(DevTable d, BeamSelect a,
                                                          const float *__restrict__ gmax,
                                                          const double2 *__restrict__ part,
                                                          int chunks)
{
    static_assert(kPickWaves * FA_BEAM_MAX == kPickThreads, "a thread per candidate slot");
    __shared__ double sh_lse[FA_BEAM_MAX];
    __shared__ double sh_key[kPickThreads];
    __shared__ uint32_t sh_id[kPickThreads];
    __shared__ int sh_cnt[kPickWaves];
    __shared__ double sel_key[FA_BEAM_MAX];
    __shared__ uint32_t sel_id[FA_BEAM_MAX];
    __shared__ uint32_t sh_mask[kPickWaves][kMaskWords];
    __shared__ int sh_bad;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nG = beam_grans(d.V), W = (d.S + 31) / 32, Kin = a.Kin, K = a.K;
    const int row0 = b * Kin;
    const bool flagged = a.status[b] != 0;
    if (tid == 0) sh_bad = 0;
    if (tid < kPickWaves) sh_cnt[tid] = 0;
    __syncthreads();
    int n = 0;
    if (!flagged) {
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
                if (bad) atomicOr(&sh_bad, 1);
            }
        }
        __syncthreads();
        // the K granules with the largest keys
        {
            double key[RG];
            bool bad = false;
#pragma unroll
            for (int r = 0; r < RG; ++r) {
                const int i = r * kPickThreads + tid;
                key[r] = -INFINITY;
                if (i < Kin * nG) {
                    const int k = i / nG;
                    const double sc = a.scores_in[row0 + k], lse = sh_lse[k];
                    if (sc > -INFINITY && lse > -INFINITY) {
                        const double x = gmax[(size_t)row0 * nG + i];
                        bad |= MODE == FA_BEAM_PROBS && x != x;
                        if (x > -INFINITY) key[r] = MODE == FA_BEAM_PROBS ? sc + log(x) : sc + (x - lse);
                    }
                }
            }
            if (bad) atomicOr(&sh_bad, 1);
            const int c = wave_topk(key, [&](int r) { return (uint32_t)(r * kPickThreads + tid); },
                                    K, sh_key + wave * FA_BEAM_MAX, sh_id + wave * FA_BEAM_MAX, lane);
            if (lane == 0) sh_cnt[wave] = c;
        }
        const int ng = block_rank(sh_key, sh_id, sh_cnt, K, sel_key, sel_id);
        // their tokens; none before the last of K granule maxima is lost
        const double floor_key = ng == K ? sel_key[K - 1] : -INFINITY;
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
                    const int i = sel_id[q], k = i / nG, g = i % nG;
                    allowed_mask(d, set_of(a, row0 + k, W), W, a.reach, g, 1, sh_mask[wave], lane);
                    const uint32_t ok = (sh_mask[wave][lane / 4] >> (8 * (lane & 3))) & 255u;
                    const int v0 = g * kBeamGran + lane * 8;
                    float x[8];
                    load8(row_of<T>(a, row0 + k), min(v0, d.V), d.V, x);
                    const double sc = a.scores_in[row0 + k], lse = sh_lse[k];
                    base[r] = (uint32_t)k * (uint32_t)d.V + (uint32_t)v0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        double kk = -INFINITY;
                        if (((ok >> j) & 1u) && x[j] > -INFINITY)
                            kk = MODE == FA_BEAM_PROBS ? sc + log((double)x[j]) : sc + ((double)x[j] - lse);
                        if (kk >= floor_key) key[r * 8 + j] = kk;
                    }
                }
            }
            __syncthreads();
            const int c = wave_topk(key, [&](int r) { return base[r / 8] + (uint32_t)(r % 8); }, K,
                                    sh_key + wave * FA_BEAM_MAX, sh_id + wave * FA_BEAM_MAX, lane);
            if (lane == 0) sh_cnt[wave] = c;
        }
        n = block_rank(sh_key, sh_id, sh_cnt, K, sel_key, sel_id);
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
        const int k = live ? (int)(sel_id[j] / (uint32_t)d.V) : j % Kin;
        const int v = live ? (int)(sel_id[j] % (uint32_t)d.V) : -1;
        if (lane == 0) {
            a.scores[o] = live ? (float)sel_key[j] : -INFINITY;
            a.tokens[o] = v;
            a.parents[o] = k;
        }
    }
    __syncthreads();
    for (int j = wave; j < n; j += kPickWaves) {
        uint32_t *to = a.states + ((size_t)b * K + j) * W;
        const int k = (int)(sel_id[j] / (uint32_t)d.V), v = (int)(sel_id[j] % (uint32_t)d.V);
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

template <class T, int MODE, int NG>
int scan(const DevTable &d, const BeamSelect &a, float *gmax, double2 *part, hipStream_t st)
{
    const int64_t waves = (beam_grans(d.V) + NG - 1) / NG;
    const int64_t nblk = (waves + kScanWaves - 1) / kScanWaves;
    const int64_t blocks = nblk * a.B * a.Kin;
    if (blocks > 0x7fffffff) return -1;
    beam_scan<T, MODE, NG><<<(unsigned)blocks, kScanWaves * kWave, 0, st>>>(d, a, gmax, part, (int)nblk);
    return (int)hipGetLastError();
}

template <class T, int MODE, int RG, int RT>
int pick(const DevTable &d, const BeamSelect &a, const float *gmax, const double2 *part, int chunks,
         hipStream_t st)
{
    beam_pick<T, MODE, RG, RT><<<a.B, kPickThreads, 0, st>>>(d, a, gmax, part, chunks);
    return (int)hipGetLastError();
}

template <class T, int MODE, int RG>
int pick_tokens(const DevTable &d, const BeamSelect &a, const float *gmax, const double2 *part,
                int chunks, hipStream_t st)
{
    if (a.K <= kPickWaves) return pick<T, MODE, RG, 1>(d, a, gmax, part, chunks, st);
    return pick<T, MODE, RG, 4>(d, a, gmax, part, chunks, st);
}

template <class T, int MODE>
int select(const DevTable &d, const BeamSelect &a, float *gmax, double2 *part, hipStream_t st)
{
    constexpr int NG = 4;
    if (int e = scan<T, MODE, NG>(d, a, gmax, part, st)) return e;
    const int nG = beam_grans(d.V), chunks = (nG + NG - 1) / NG;
    if (a.Kin * nG <= 4 * kPickThreads) return pick_tokens<T, MODE, 4>(d, a, gmax, part, chunks, st);
    return pick_tokens<T, MODE, 32>(d, a, gmax, part, chunks, st);
}

template <class T>
int select_mode(const DevTable &d, const BeamSelect &a, float *gmax, double2 *part, hipStream_t st)
{
    return a.mode == FA_BEAM_LOGITS ? select<T, FA_BEAM_LOGITS>(d, a, gmax, part, st)
                                    : select<T, FA_BEAM_PROBS>(d, a, gmax, part, st);
}

}  // namespace

BeamWs beam_ws_layout(const HostTable &t, int32_t B, int32_t Kin)
{
    auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t n = (size_t)B * Kin * beam_grans(t.V);
    BeamWs w;
    w.gmax = 0;
    w.part = al(n * sizeof(float));
    w.total = al(w.part + n * 2 * sizeof(double));
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
    float *gmax = reinterpret_cast<float *>(ws + w.gmax);
    double2 *part = reinterpret_cast<double2 *>(ws + w.part);
    hipStream_t st = (hipStream_t)stream;
    if (a.dtype == FA_F32) return select_mode<float>(d, a, gmax, part, st);
    if (a.dtype == FA_F16) return select_mode<_Float16>(d, a, gmax, part, st);
    return select_mode<Bf16>(d, a, gmax, part, st);
}

}  // namespace fa
