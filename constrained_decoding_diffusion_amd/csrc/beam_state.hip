// Per-hypothesis memory of a beam search: slots of caches moved after the
// chosen parents, and the hypotheses read back from the recorded steps.
#include <algorithm>

#include "device_common.h"

namespace fa {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kMoveItems = 24;  // items of one launch: their descriptors travel as kernel arguments
constexpr int kUnit = 16;       // bytes a thread moves per slot

struct MoveItem {
    const char *src;
    char *dst;
    int64_t sb, sk, sr, db, dk, dr;  // batch, slot and row strides
    int64_t row_bytes;
    uint32_t per_row;  // units of a row, its last one shorter when 16 does not divide it
    uint32_t units;    // of a slot
    uint32_t blocks;   // workgroups of a batch row
    uint32_t first;    // first workgroup of the item
};
struct MoveArgs {
    int32_t n, B, K;
    const int32_t *parents;
    MoveItem it[kMoveItems];
};
static_assert(sizeof(MoveArgs) <= 4096, "kernel arguments");

template <class T>
__device__ inline T load_as(const char *p)
{
    T x;
    __builtin_memcpy(&x, p, sizeof(T));  // any alignment
    return x;
}

// One thread: one unit of every slot of a batch row.  All slots are loaded
// before any is stored, and no other thread touches these bytes, so the
// permutation needs no second buffer whatever the parents are.
template <int KMAX>
__global__ __launch_bounds__(kMoveThreads) void beam_move(MoveArgs a)
{
    int i = 0;
    while (i + 1 < a.n && blockIdx.x >= a.it[i + 1].first) ++i;
    const MoveItem &m = a.it[i];
    const uint32_t blk = blockIdx.x - m.first;
    const int b = blk / m.blocks;
    const uint32_t u = (blk % m.blocks) * kMoveThreads + threadIdx.x;
    if (u >= m.units) return;
    const uint32_t r = u / m.per_row, c = u % m.per_row;
    const char *src = m.src + (int64_t)b * m.sb + (int64_t)r * m.sr + (int64_t)c * kUnit;
    char *dst = m.dst + (int64_t)b * m.db + (int64_t)r * m.dr + (int64_t)c * kUnit;
    const int left = (int)min((int64_t)kUnit, m.row_bytes - (int64_t)c * kUnit);
    const bool in_place = m.src == m.dst;
    const int32_t *par = a.parents + (size_t)b * a.K;
    uint4 x[KMAX];
    if (left == kUnit) {
#pragma unroll
        for (int k = 0; k < KMAX; ++k) {
            if (k >= a.K) continue;
            int p = par[k];
            if (p < 0 || p >= a.K) p = k;
            if (in_place && p == k) continue;
            x[k] = load_as<uint4>(src + p * m.sk);
        }
#pragma unroll
        for (int k = 0; k < KMAX; ++k) {
            if (k >= a.K) continue;
            int p = par[k];
            if (p < 0 || p >= a.K) p = k;
            if (in_place && p == k) continue;
            __builtin_memcpy(dst + k * m.dk, &x[k], kUnit);
        }
    } else {
        // the short last unit of a row, byte by byte
        for (int j = 0; j < left; ++j) {
            uint8_t y[KMAX];
#pragma unroll
            for (int k = 0; k < KMAX; ++k) {
                if (k >= a.K) continue;
                int p = par[k];
                if (p < 0 || p >= a.K) p = k;
                if (in_place && p == k) continue;
                y[k] = (uint8_t)src[p * m.sk + j];
            }
#pragma unroll
            for (int k = 0; k < KMAX; ++k) {
                if (k >= a.K) continue;
                int p = par[k];
                if (p < 0 || p >= a.K) p = k;
                if (in_place && p == k) continue;
                dst[k * m.dk + j] = (char)y[k];
            }
        }
    }
}

// One workgroup: one batch row, a thread per hypothesis walking back.
__global__ __launch_bounds__(FA_BEAM_MAX) void beam_walk(int T, int B, int K,
                                                         const int32_t *__restrict__ tokens,
                                                         const int32_t *__restrict__ parents,
                                                         int32_t *__restrict__ out)
{
    const int b = blockIdx.x, k = threadIdx.x;
    if (k >= K) return;
    int j = k;
    for (int t = T - 1; t >= 0; --t) {
        const size_t o = ((size_t)t * B + b) * K;
        const bool ok = j >= 0 && j < K;
        out[((size_t)b * K + k) * T + t] = ok ? tokens[o + j] : -1;
        if (ok) j = parents[o + j];
    }
}

}  // namespace

int launch_beam_reorder(const fa_beam_item *items, int n, int B, int K, const int32_t *parents,
                        void *stream)
{
    hipStream_t st = (hipStream_t)stream;
    // every item must fit before the first is launched
    for (int i = 0; i < n; ++i) {
        const fa_beam_item &x = items[i];
        const int64_t per_row = x.row_bytes / kUnit + (x.row_bytes % kUnit != 0);
        if (x.rows == 0 || per_row == 0) continue;
        if (per_row > 0xffffffffLL || x.rows > 0xffffffffLL / per_row) return -1;
        const int64_t blocks = (x.rows * per_row + kMoveThreads - 1) / kMoveThreads;
        if (blocks * B > 0x7fffffffLL) return -1;
    }
    MoveArgs a;
    a.B = B;
    a.K = K;
    a.parents = parents;
    for (int i = 0; i < n;) {
        a.n = 0;
        int64_t blocks = 0;
        for (; i < n && a.n < kMoveItems; ++i) {
            const fa_beam_item &x = items[i];
            if (x.rows == 0 || x.row_bytes == 0) continue;
            MoveItem &m = a.it[a.n];
            m.src = static_cast<const char *>(x.src);
            m.dst = static_cast<char *>(x.dst);
            m.sb = x.src_batch_stride;
            m.sk = x.src_beam_stride;
            m.sr = x.src_row_stride;
            m.db = x.dst_batch_stride;
            m.dk = x.dst_beam_stride;
            m.dr = x.dst_row_stride;
            m.row_bytes = x.row_bytes;
            m.per_row = (uint32_t)((x.row_bytes + kUnit - 1) / kUnit);
            m.units = (uint32_t)(x.rows * m.per_row);
            m.blocks = (m.units + (uint64_t)kMoveThreads - 1) / kMoveThreads;
            m.first = (uint32_t)blocks;
            if (blocks + (int64_t)m.blocks * B > 0x7fffffffLL) break;
            blocks += (int64_t)m.blocks * B;
            ++a.n;
        }
        if (a.n == 0) continue;
        const unsigned g = (unsigned)blocks;
        if (K <= 4) beam_move<4><<<g, kMoveThreads, 0, st>>>(a);
        else if (K <= 8) beam_move<8><<<g, kMoveThreads, 0, st>>>(a);
        else if (K <= 16) beam_move<16><<<g, kMoveThreads, 0, st>>>(a);
        else if (K <= 32) beam_move<32><<<g, kMoveThreads, 0, st>>>(a);
        else beam_move<64><<<g, kMoveThreads, 0, st>>>(a);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return (int)e;
    }
    return 0;
}

int launch_beam_trace(int T, int B, int K, const int32_t *tokens, const int32_t *parents,
                      int32_t *out, void *stream)
{
    beam_walk<<<B, FA_BEAM_MAX, 0, (hipStream_t)stream>>>(T, B, K, tokens, parents, out);
    return (int)hipGetLastError();
}

}  // namespace fa
