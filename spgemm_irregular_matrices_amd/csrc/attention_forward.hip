// Softmax attention over the entries of a CSR mask, forward.
#include "attention.h"

namespace sg {

namespace {

constexpr int kWaves = 4;  // wavefronts per work group; each has a piece of its own

// Half precision keeps only 2^-24 absolutely: probabilities are held times
// 2^14 there, so that the many small ones of a long row keep their 11 bits
// (the largest is 2^14, a quarter of the type's range). The sum carries the
// same factor.
template <class T>
constexpr float kProbShift = std::is_same<T, _Float16>::value ? 14.f : 0.f;

// One wavefront: the 16 query heads [16*mt, 16*mt+16) of a key head's group
// against the piece's keys, one tile of KT gathered keys after another.
template <class G, class T>
__global__ __launch_bounds__(kWaves* kWave) void k_attn_forward(ForwardArgs a) {
    const int lane = lane_id();
    const int64_t unit = xcd_block() * kWaves + threadIdx.x / kWave;
    const int64_t npieces = a.side.npieces;
    if (unit >= npieces * a.s.hkv * a.s.mtiles) return;
    const int hm = (int)(unit / npieces);  // key head and group of 16 query heads
    const AttnPiece pc = a.side.pieces[unit - (int64_t)hm * npieces];
    const int h = hm / a.s.mtiles, mt = hm - h * a.s.mtiles;
    const int n = lane & 15;  // this lane's query head in the tile
    const int g = 16 * mt + n;
    const bool has = g < a.s.group;
    const int hq = h * a.s.group + g;
    const int row_bytes = a.s.dim * (int)sizeof(T);

    typename G::RowFrag q;
    G::zero_row(q);
    if (has) G::load_row(a.q.base + pc.row * a.q.row + hq * a.q.head, row_bytes, q);
    typename G::Acc o;
    G::zero_acc(o);
    float m = -INFINITY, l = 0.f;  // l: this lane's keys only, until the end

    const char* kb = a.k.base + h * a.k.head;
    const char* vb = a.v.base + h * a.v.head;
    const int32_t* idx = a.side.idx + pc.first;
    for (int t0 = 0; t0 < pc.len; t0 += G::KT) {
        const int left = pc.len - t0;
        // lanes past the end repeat the last entry: every address is one the row names
        const uint32_t id = (uint32_t)idx[t0 + min(lane & (G::KT - 1), left - 1)];
        const uint32_t ko = id * a.k.unit, vo = id * a.v.unit;

        f32x4 s[G::KSUB];
#pragma unroll
        for (int b = 0; b < G::KSUB; ++b) {
            const uint32_t off = __shfl(ko, 16 * b + n, kWave);
            typename G::RowFrag k;
            G::load_row(kb + ((uint64_t)off << a.k.shift), row_bytes, k);
            s[b] = G::dot(k, q, f32x4{0, 0, 0, 0});
        }
        float p[G::VK], top = -INFINITY;
#pragma unroll
        for (int j = 0; j < G::VK; ++j) {
            p[j] = G::key_of(j) < left ? s[j >> 2][j & 3] * a.s.c : -INFINITY;
            top = fmaxf(top, p[j]);
        }
        const float mn = fmaxf(m, quad_max(top));
        const float ms = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: weights 0, not NaN
        const float fix = fast_exp2(m - ms);
        m = mn;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < G::VK; ++j) {
            p[j] = fast_exp2(p[j] - (ms - kProbShift<T>));
            sum += p[j];
        }
        l = l * fix + sum;
        G::scale_acc(o, fix);
        typename G::Probs pr;
        G::pack_probs(p, pr);
#pragma unroll
        for (int u = 0; u < G::U; ++u) {
            typename G::VBlock v;
#pragma unroll
            for (int j = 0; j < G::VK; ++j) {
                const uint32_t off = __shfl(vo, G::key_of(j), kWave);
                G::load_chunk(vb + ((uint64_t)off << a.v.shift), u, row_bytes, v.w[j]);
                if (G::key_of(j) >= left) {  // 0 weight times what the row holds may be NaN
#pragma unroll
                    for (int i = 0; i < G::VW; ++i) v.w[j][i] = 0;
                }
            }
            G::accumulate(v, pr, u, o);
        }
    }
    l = quad_sum(l);
    if (!has) return;
    if (pc.slot < 0) {
        const float f = l == 0.f ? 0.f : 1.f / l;
        char* row = a.out.base + pc.row * a.out.row + hq * a.out.head;
#pragma unroll
        for (int u = 0; u < G::U; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) G::store_out(o, u, r, f, row, row_bytes);
        if (a.lse && lane < 16)
            a.lse[(int64_t)pc.row * a.s.hq + hq] =
                l == 0.f ? -INFINITY : (m - kProbShift<T> + fast_log2(l)) * kLn2;
    } else {
        const int64_t at = (int64_t)pc.slot * a.s.hq + hq;
        float* dst = a.part + at * a.s.dim;
#pragma unroll
        for (int u = 0; u < G::U; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) G::store_part(o, u, r, 1.f, dst, a.s.dim);
        if (lane < 16) {
            a.part_ml[2 * at] = m;
            a.part_ml[2 * at + 1] = l;
        }
    }
}

// The rows of more than one piece: one wavefront per row and query head
// joins the pieces, in their order.
template <class T>
__global__ __launch_bounds__(kWaves* kWave) void k_attn_join(ForwardArgs a) {
    const int lane = lane_id();
    const int64_t unit = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
    if (unit >= a.side.nsplits * a.s.hq) return;
    const int64_t sp = unit / a.s.hq;
    const int hq = (int)(unit - sp * a.s.hq);
    const AttnSplit s = a.side.splits[sp];
    float m = -INFINITY;
    for (int i = lane; i < s.count; i += kWave)
        m = fmaxf(m, a.part_ml[2 * ((int64_t)(s.slot + i) * a.s.hq + hq)]);
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, kWave));
    const float ms = m == -INFINITY ? 0.f : m;
    float l = 0.f, o[SPGEMM_ATTENTION_MAX_HEAD_DIM / kWave] = {};
    for (int i = 0; i < s.count; ++i) {
        const int64_t at = (int64_t)(s.slot + i) * a.s.hq + hq;
        const float w = fast_exp2(a.part_ml[2 * at] - ms);
        l += a.part_ml[2 * at + 1] * w;
        const float* src = a.part + at * a.s.dim;
#pragma unroll
        for (int j = 0; j < SPGEMM_ATTENTION_MAX_HEAD_DIM / kWave; ++j)
            if (j * kWave + lane < a.s.dim) o[j] += src[j * kWave + lane] * w;
    }
    const float f = l == 0.f ? 0.f : 1.f / l;
    T* dst = reinterpret_cast<T*>(a.out.base + s.row * a.out.row + hq * a.out.head);
#pragma unroll
    for (int j = 0; j < SPGEMM_ATTENTION_MAX_HEAD_DIM / kWave; ++j)
        if (j * kWave + lane < a.s.dim) dst[j * kWave + lane] = (T)(o[j] * f);
    if (a.lse && lane == 0)
        a.lse[(int64_t)s.row * a.s.hq + hq] =
            l == 0.f ? -INFINITY : (m - kProbShift<T> + fast_log2(l)) * kLn2;
}

}  // namespace

void attention_forward(const ForwardArgs& a, hipStream_t st) {
    const int64_t units = a.side.npieces * a.s.hkv * a.s.mtiles;
    if (units == 0) return;
    with_type(a.s.type, a.s.dim, [&](auto tag) {
        using Tag = decltype(tag);
        auto run = k_attn_forward<typename Tag::Geo, typename Tag::Elem>;
        hipLaunchKernelGGL(run, dim3(grid_1d(xcd_grid(ceil_div(units, kWaves)))),
                           dim3(kWaves * kWave), 0, st, a);
        SG_LAUNCH_CHECK();
        if (a.side.nsplits > 0) {
            hipLaunchKernelGGL(k_attn_join<typename Tag::Elem>,
                               dim3(grid_1d(ceil_div(a.side.nsplits * a.s.hq, kWaves))),
                               dim3(kWaves * kWave), 0, st, a);
            SG_LAUNCH_CHECK();
        }
    });
}

}  // namespace sg
