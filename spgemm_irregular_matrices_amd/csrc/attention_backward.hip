// Gradients of softmax attention over the entries of a CSR mask. The
// probabilities are recomputed twice from q, k and the log-sum-exp: once row
// by row for dq, once column by column for dk and dv. No pass adds to memory
// that another work group adds to, so nothing depends on the order of work
// groups and no buffer has to be cleared.
#include "attention.h"

namespace sg {

namespace {

constexpr int kWaves = 4;

// Half precision: dS is scaled by a power of two that follows its largest
// magnitude so far (about 2^11 for that one), as the running maximum of a
// softmax does, because gradients can lie anywhere in the floats' range while
// the type ends at 65504 and loses bits below 2^-14. Values that are small
// beside the largest lose nothing that the sum would keep.
struct HalfScale {
    float s = 0x1p60f;
    // The factor for sums made so far, after admitting magnitude mx (alike
    // in all lanes whose sums share a column).
    __device__ __forceinline__ float admit(float mx) {
        if (!(mx * s > 32768.f) || !(mx < INFINITY)) return 1.f;
        const int e = (int)(__builtin_bit_cast(uint32_t, mx) >> 23) - 127;
        const float to = __builtin_bit_cast(float, (uint32_t)(127 + 11 - e) << 23);
        const float f = to / s;
        s = to;
        return f;
    }
};
// Probabilities of a half-precision dv: times 2^14, as in the forward pass.
template <class T>
constexpr float kProbScale = std::is_same<T, _Float16>::value ? 0x1p14f : 1.f;

// dq: one wavefront per piece of a row and 16 query heads of a key head, as
// in the forward pass. S^T and dP^T = V dO^T come from the same gathered rows
// in the same layout, dQ^T += K^T dS^T takes K again in the chunk layout
// (the rows were read a moment before, so these loads hit the caches).
template <class G, class T>
__global__ __launch_bounds__(kWaves* kWave) void k_attn_grad_q(BackwardArgs a) {
    const int lane = lane_id();
    const int64_t unit = xcd_block() * kWaves + threadIdx.x / kWave;
    const int64_t npieces = a.rows.npieces;
    if (unit >= npieces * a.s.hkv * a.s.mtiles) return;
    const int hm = (int)(unit / npieces);
    const AttnPiece pc = a.rows.pieces[unit - (int64_t)hm * npieces];
    const int h = hm / a.s.mtiles, mt = hm - h * a.s.mtiles;
    const int n = lane & 15;
    const int g = 16 * mt + n;
    const bool has = g < a.s.group;
    const int hq = h * a.s.group + g;
    const int row_bytes = a.s.dim * (int)sizeof(T);

    typename G::RowFrag q, dout;
    G::zero_row(q);
    G::zero_row(dout);
    float lse2 = INFINITY, delta = 0.f;  // lanes without a head: weights 0
    if (has) {
        G::load_row(a.q.base + pc.row * a.q.row + hq * a.q.head, row_bytes, q);
        G::load_row(a.dout.base + pc.row * a.dout.row + hq * a.dout.head, row_bytes, dout);
        typename G::RowFrag out;
        G::load_row(a.out.base + pc.row * a.out.row + hq * a.out.head, row_bytes, out);
        delta = G::dot_lane(dout, out);
        const float x = a.lse[(int64_t)pc.row * a.s.hq + hq];
        lse2 = x == -INFINITY ? INFINITY : x * kLog2e;
    }
    delta = quad_sum(delta);
    if (has && lane < 16 && pc.lead)
        a.delta[(int64_t)pc.row * a.s.hq + hq] = delta;

    typename G::Acc o;
    G::zero_acc(o);
    HalfScale hs;
    const char* kb = a.k.base + h * a.k.head;
    const char* vb = a.v.base + h * a.v.head;
    const int32_t* idx = a.rows.idx + pc.first;
    for (int t0 = 0; t0 < pc.len; t0 += G::KT) {
        const int left = pc.len - t0;
        const uint32_t id = (uint32_t)idx[t0 + min(lane & (G::KT - 1), left - 1)];
        const uint32_t ko = id * a.k.unit, vo = id * a.v.unit;
        f32x4 s[G::KSUB], dp[G::KSUB];
#pragma unroll
        for (int b = 0; b < G::KSUB; ++b) {
            typename G::RowFrag x;
            G::load_row(kb + ((uint64_t)__shfl(ko, 16 * b + n, kWave) << a.k.shift), row_bytes, x);
            s[b] = G::dot(x, q, f32x4{0, 0, 0, 0});
            G::load_row(vb + ((uint64_t)__shfl(vo, 16 * b + n, kWave) << a.v.shift), row_bytes, x);
            dp[b] = G::dot(x, dout, f32x4{0, 0, 0, 0});
        }
        float ds[G::VK];
#pragma unroll
        for (int j = 0; j < G::VK; ++j) {
            const float p = fast_exp2(fmaf(s[j >> 2][j & 3], a.s.c, -lse2));
            ds[j] = G::key_of(j) < left ? p * (dp[j >> 2][j & 3] - delta) : 0.f;
        }
        if constexpr (std::is_same<T, _Float16>::value) {
            float mx = 0.f;
#pragma unroll
            for (int j = 0; j < G::VK; ++j) mx = fmaxf(mx, fabsf(ds[j]));
            const float f = hs.admit(quad_max(mx));
            if (__any(f != 1.f)) G::scale_acc(o, f);
#pragma unroll
            for (int j = 0; j < G::VK; ++j) ds[j] *= hs.s;
        }
        typename G::Probs pr;
        G::pack_probs(ds, pr);
#pragma unroll
        for (int u = 0; u < G::U; ++u) {
            typename G::VBlock x;
#pragma unroll
            for (int j = 0; j < G::VK; ++j) {
                const uint32_t off = __shfl(ko, G::key_of(j), kWave);
                G::load_chunk(kb + ((uint64_t)off << a.k.shift), u, row_bytes, x.w[j]);
                if (G::key_of(j) >= left) {
#pragma unroll
                    for (int i = 0; i < G::VW; ++i) x.w[j][i] = 0;
                }
            }
            G::accumulate(x, pr, u, o);
        }
    }
    if (!has) return;
    float f = a.s.scale;
    if constexpr (std::is_same<T, _Float16>::value) f /= hs.s;
    if (pc.slot < 0) {
        char* row = a.dq.base + pc.row * a.dq.row + hq * a.dq.head;
#pragma unroll
        for (int u = 0; u < G::U; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) G::store_out(o, u, r, f, row, row_bytes);
    } else {
        float* dst = a.part_q + ((int64_t)pc.slot * a.s.hq + hq) * a.s.dim;
#pragma unroll
        for (int u = 0; u < G::U; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) G::store_part(o, u, r, f, dst, a.s.dim);
    }
}

// dk and dv: one wavefront per piece of a column and key head. The gathered
// list is the (row, query head) pairs of the piece's entries, and the other
// operand is the column's one k (or v) row in all 16 places: S, dP and so P
// and dS come out alike in 16 columns, which is what lets them go straight
// into the second products; the matrix units have the room (a pair costs
// about as many cycles as its two gathered rows take to arrive).
template <class G, class T>
__global__ __launch_bounds__(kWaves* kWave) void k_attn_grad_kv(BackwardArgs a) {
    const int lane = lane_id();
    const int64_t unit = xcd_block() * kWaves + threadIdx.x / kWave;
    const int64_t npieces = a.cols.npieces;
    if (unit >= npieces * a.s.hkv) return;
    const int h = (int)(unit / npieces);
    const AttnPiece pc = a.cols.pieces[unit - (int64_t)h * npieces];
    const int n = lane & 15;
    const int row_bytes = a.s.dim * (int)sizeof(T);
    constexpr bool half = std::is_same<T, _Float16>::value;

    typename G::RowFrag k, v;
    G::load_row(a.krow.base + pc.row * a.krow.row + h * a.krow.head, row_bytes, k);
    G::load_row(a.vrow.base + pc.row * a.vrow.row + h * a.vrow.head, row_bytes, v);
    typename G::Acc dk, dv;
    G::zero_acc(dk);
    G::zero_acc(dv);
    HalfScale hs;
    const char* qb = a.gq.base + (int64_t)h * a.s.group * a.gq.head;
    const char* gb = a.gdout.base + (int64_t)h * a.s.group * a.gdout.head;
    const uint32_t qhead = (uint32_t)(a.gq.head >> a.gq.shift);
    const uint32_t ghead = (uint32_t)(a.gdout.head >> a.gdout.shift);
    const int32_t* idx = a.cols.idx + pc.first;
    const int64_t pairs = (int64_t)pc.len * a.s.group;
    for (int64_t t0 = 0; t0 < pairs; t0 += G::KT) {
        const int left = (int)min(pairs - t0, (int64_t)G::KT);
        const uint32_t x = (uint32_t)t0 + min(lane & (G::KT - 1), left - 1);
        const uint32_t e = a.group_div.div(x), g = x - e * a.s.group;
        const uint32_t id = (uint32_t)idx[e];
        const uint32_t qo = id * a.gq.unit + g * qhead, go = id * a.gdout.unit + g * ghead;
        const int64_t at = (int64_t)id * a.s.hq + h * a.s.group + g;
        const float lse = a.lse[at], dl = a.delta[at];
        const float lse2 = lse == -INFINITY ? INFINITY : lse * kLog2e;
        f32x4 s[G::KSUB], dp[G::KSUB];
#pragma unroll
        for (int b = 0; b < G::KSUB; ++b) {
            typename G::RowFrag f;
            G::load_row(qb + ((uint64_t)__shfl(qo, 16 * b + n, kWave) << a.gq.shift), row_bytes, f);
            s[b] = G::dot(f, k, f32x4{0, 0, 0, 0});
            G::load_row(gb + ((uint64_t)__shfl(go, 16 * b + n, kWave) << a.gdout.shift), row_bytes,
                        f);
            dp[b] = G::dot(f, v, f32x4{0, 0, 0, 0});
        }
        float p[G::VK], ds[G::VK];
#pragma unroll
        for (int j = 0; j < G::VK; ++j) {
            const float l2 = __shfl(lse2, G::key_of(j), kWave);
            const float dj = __shfl(dl, G::key_of(j), kWave);
            const bool on = G::key_of(j) < left;
            p[j] = on ? fast_exp2(fmaf(s[j >> 2][j & 3], a.s.c, -l2)) : 0.f;
            ds[j] = on ? p[j] * (dp[j >> 2][j & 3] - dj) : 0.f;
            p[j] *= kProbScale<T>;
        }
        if constexpr (half) {
            float mx = 0.f;
#pragma unroll
            for (int j = 0; j < G::VK; ++j) mx = fmaxf(mx, fabsf(ds[j]));
            const float f = hs.admit(quad_max(mx));
            if (__any(f != 1.f)) G::scale_acc(dk, f);
#pragma unroll
            for (int j = 0; j < G::VK; ++j) ds[j] *= hs.s;
        }
        typename G::Probs pp, pd;
        G::pack_probs(p, pp);
        G::pack_probs(ds, pd);
#pragma unroll
        for (int u = 0; u < G::U; ++u) {
            typename G::VBlock c;
#pragma unroll
            for (int j = 0; j < G::VK; ++j) {
                const uint32_t off = __shfl(go, G::key_of(j), kWave);
                G::load_chunk(gb + ((uint64_t)off << a.gdout.shift), u, row_bytes, c.w[j]);
                if (G::key_of(j) >= left) {
#pragma unroll
                    for (int i = 0; i < G::VW; ++i) c.w[j][i] = 0;
                }
            }
            G::accumulate(c, pp, u, dv);
#pragma unroll
            for (int j = 0; j < G::VK; ++j) {
                const uint32_t off = __shfl(qo, G::key_of(j), kWave);
                G::load_chunk(qb + ((uint64_t)off << a.gq.shift), u, row_bytes, c.w[j]);
                if (G::key_of(j) >= left) {
#pragma unroll
                    for (int i = 0; i < G::VW; ++i) c.w[j][i] = 0;
                }
            }
            G::accumulate(c, pd, u, dk);
        }
    }
    float fk = a.s.scale;
    if constexpr (half) fk /= hs.s;
    const float fv = 1.f / kProbScale<T>;
    // the 16 columns are alike: column r stores register r
    char* krow = a.dk.base + pc.row * a.dk.row + h * a.dk.head;
    char* vrow = a.dv.base + pc.row * a.dv.row + h * a.dv.head;
    float* part =
        pc.slot < 0 ? nullptr : a.part_kv + ((int64_t)pc.slot * a.s.hkv + h) * 2 * a.s.dim;
#pragma unroll
    for (int u = 0; u < G::U; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (n != r) continue;
            if (part) {
                G::store_part(dk, u, r, fk, part, a.s.dim);
                G::store_part(dv, u, r, fv, part + a.s.dim, a.s.dim);
            } else {
                G::store_out(dk, u, r, fk, krow, row_bytes);
                G::store_out(dv, u, r, fv, vrow, row_bytes);
            }
        }
}

// The rows of more than one piece: the sum of the pieces, in their order.
// One wavefront per row, head and output (`outs` of them side by side).
template <class T>
__global__ __launch_bounds__(kWaves* kWave) void k_attn_join_sum(AttnSide side, const float* part,
                                                                 int heads, int outs, int dim,
                                                                 AttnRows out0, AttnRows out1) {
    const int lane = lane_id();
    const int64_t unit = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
    if (unit >= side.nsplits * heads * outs) return;
    const int64_t sp = unit / (heads * outs);
    const int ho = (int)(unit - sp * heads * outs);
    const int h = ho / outs;
    const AttnSplit s = side.splits[sp];
    float x[SPGEMM_ATTENTION_MAX_HEAD_DIM / kWave] = {};
    for (int i = 0; i < s.count; ++i) {
        const float* src = part + ((int64_t)(s.slot + i) * heads * outs + ho) * dim;
#pragma unroll
        for (int j = 0; j < SPGEMM_ATTENTION_MAX_HEAD_DIM / kWave; ++j)
            if (j * kWave + lane < dim) x[j] += src[j * kWave + lane];
    }
    const AttnRows& o = ho - h * outs ? out1 : out0;
    T* dst = reinterpret_cast<T*>(o.base + s.row * o.row + h * o.head);
#pragma unroll
    for (int j = 0; j < SPGEMM_ATTENTION_MAX_HEAD_DIM / kWave; ++j)
        if (j * kWave + lane < dim) dst[j * kWave + lane] = (T)x[j];
}

template <class T>
void join_sum(const AttnSide& side, const float* part, int heads, int outs, int dim,
              const AttnRows& out0, const AttnRows& out1, hipStream_t st) {
    if (side.nsplits == 0) return;
    hipLaunchKernelGGL(k_attn_join_sum<T>,
                       dim3(grid_1d(ceil_div(side.nsplits * heads * outs, kWaves))),
                       dim3(kWaves * kWave), 0, st, side, part, heads, outs, dim, out0, out1);
    SG_LAUNCH_CHECK();
}

}  // namespace

void attention_backward(const BackwardArgs& a, hipStream_t st) {
    with_type(a.s.type, a.s.dim, [&](auto tag) {
        using Tag = decltype(tag);
        using T = typename Tag::Elem;
        const int64_t rows = a.rows.npieces * a.s.hkv * a.s.mtiles;
        if (rows > 0) {
            auto run = k_attn_grad_q<typename Tag::Geo, T>;
            hipLaunchKernelGGL(run, dim3(grid_1d(xcd_grid(ceil_div(rows, kWaves)))),
                               dim3(kWaves * kWave), 0, st, a);
            SG_LAUNCH_CHECK();
            join_sum<T>(a.rows, a.part_q, a.s.hq, 1, a.s.dim, a.dq, a.dq, st);
        }
        const int64_t cols = a.cols.npieces * a.s.hkv;
        if (cols > 0) {
            auto run = k_attn_grad_kv<typename Tag::Geo, T>;
            hipLaunchKernelGGL(run, dim3(grid_1d(xcd_grid(ceil_div(cols, kWaves)))),
                               dim3(kWaves * kWave), 0, st, a);
            SG_LAUNCH_CHECK();
            join_sum<T>(a.cols, a.part_kv, a.s.hkv, 2, a.s.dim, a.dk, a.dv, st);
        }
    });
}

}  // namespace sg
