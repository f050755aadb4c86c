// Training side of the router: its load and losses (edge_moe_balance) and its
// backward pass (edge_moe_route_backward).
//
// With z the logits of a token, p = softmax(z) over all E experts, lse = log sum
// exp z, and for each sequence s of n_s tokens c_se = picks of expert e,
// f_se = E / (k n_s) c_se, P_se = mean of p_te over the sequence:
//   balance loss  L_b = 1/S' sum over the S' sequences with tokens of sum_e f_se P_se
//   z loss        L_z = 1/n sum over their n tokens of lse_t^2
// The counts are constants to the gradient, so with g_b, g_z the losses'
// gradients and w = softmax over the selected logits:
//   dz_te =  g_b / (S' n_s) p_te (f_se - sum_i p_ti f_si)  +  2 g_z / n lse_t p_te
//          + sum_{j: idx_tj = e} w_tj (dw_tj - sum_i w_ti dw_ti)
//   dx = dz W_r,   dW_r = dz^T x,   dbias = sum_t dz
//
// Kernels:
//   rt_load         softmax rows of a chunk of tokens, column sums and counts
//   rt_load_reduce  chunks added in order (float64) per sequence; the losses
//   rt_dlogits      dz by rows, float32 and / or as three bf16 planes
//   rt_products     dx and dW_r on the bf16 matrix cores: dz is the exact sum of
//                   its planes (hi + mid + lo: 24 bits), x and W_r are bf16, every
//                   product is exact in float32 and the sums are float32; and dbias,
//                   the chunks of rt_dlogits added in order
//   rt_finish       the slices of dW_r and dx added in order
#include "common.h"
#include "lds_load.h"
#include "operators.h"

namespace em {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Tokens per workgroup of rt_load and rt_dlogits, one or four a wave (whose aligned
// rows are all asked for at once): few enough that small batches spread over the
// compute units, where the chain of one token's reductions is what takes the time.
constexpr int WT = 4;          // tokens a wave takes at most
int load_chunk(int T) { return T <= 2048 ? 4 : 4 * WT; }
int grad_chunk(int T) { return T <= 4096 ? 4 : 4 * WT; }

// ---- wave reductions: DPP within rows of 16 lanes, two broadcasts across them
// (no LDS); the same value in every lane.
template <int CTRL, int ROWS>
EM_DEV float dpp_f(float v, float old) {
    return __uint_as_float(__builtin_amdgcn_update_dpp((int)__float_as_uint(old), (int)__float_as_uint(v), CTRL, ROWS, 0xF, false));
}
EM_DEV float lane63(float v) { return __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(v), 63)); }

EM_DEV float wave_max(float v) {
    v = fmaxf(v, dpp_f<0xB1, 0xF>(v, v));        // quad_perm [1,0,3,2], [2,3,0,1]
    v = fmaxf(v, dpp_f<0x4E, 0xF>(v, v));
    v = fmaxf(v, dpp_f<0x141, 0xF>(v, v));       // row_half_mirror, row_mirror
    v = fmaxf(v, dpp_f<0x140, 0xF>(v, v));
    v = fmaxf(v, dpp_f<0x142, 0xA>(v, v));       // row_bcast:15, :31: lane 63 has seen every row
    v = fmaxf(v, dpp_f<0x143, 0xC>(v, v));
    return lane63(v);
}
EM_DEV float wave_sum(float v) {
    v += dpp_f<0xB1, 0xF>(v, 0.f);
    v += dpp_f<0x4E, 0xF>(v, 0.f);
    v += dpp_f<0x141, 0xF>(v, 0.f);
    v += dpp_f<0x140, 0xF>(v, 0.f);
    v += dpp_f<0x142, 0xA>(v, 0.f);
    v += dpp_f<0x143, 0xC>(v, 0.f);
    return lane63(v);
}

// A wave's own LDS accesses complete in order; this keeps the compiler from
// reordering those of different lanes to one place.
EM_DEV void wave_lds_order() {
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
}

// ---- sequences -----------------------------------------------------------------
// Tokens [lo(s), hi(s)) of sequence s; offsets outside 0..T or descending are
// clamped, so that no token outside 0..T-1 is named.
struct Seqs {
    const int32_t* off;
    int S, T;
    EM_DEV int lo(int s) const { return off ? min(max(off[s], 0), T) : 0; }
    EM_DEV int hi(int s) const { return off ? min(max(off[s + 1], lo(s)), T) : T; }
};

// First sequence that can hold token t: the last one that starts at or before
// it (0 if none does).  64 offsets a step: two rounds of loads up to S = 4095.
EM_DEV int find_seq(const Seqs& q, int t) {
    if (!q.off) return 0;
    const int lane = lane_id();
    int base = 0;
    if (q.S >= 64) {
        const int n = __popcll(__ballot(64 * lane <= q.S && q.off[min(64 * lane, q.S)] <= t));
        base = 64 * max(n - 1, 0);
    }
    const int n = __popcll(__ballot(base + lane <= q.S && q.off[min(base + lane, q.S)] <= t));
    return min(max(base + n - 1, 0), q.S - 1);
}

// Sequences with tokens, and their tokens.
EM_DEV void live_seqs(const Seqs& q, int& live, int& tokens) {
    if (!q.off) {
        live = 1;
        tokens = q.T;
        return;
    }
    int l = 0, n = 0;
    for (int s = lane_id(); s < q.S; s += 64) {
        const int c = q.hi(s) - q.lo(s);
        l += c > 0;
        n += c;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        l += __shfl_xor(l, o, 64);
        n += __shfl_xor(n, o, 64);
    }
    live = l;
    tokens = n;
}

// ---- logit rows ----------------------------------------------------------------
// A wave holds a row: lane l has experts 256 i + 4 l + c (c < 4).  Experts past
// E read as -infinity (probability 0).  Rows that are not 16-byte aligned (E no
// multiple of 4) arrive as 64 neighbours a load, expert 256 i + 64 c + l, and are
// turned through the wave's LDS row (loads of every fourth expert took 44 us for
// load and gradient of 14311 x 399, 35 this way).  Both forms in one kernel cost the
// unaligned one: the compiler waits for the loads before at each 256 experts of it.
template <int NV>
EM_DEV void load_row(float (&v)[NV][4], const float* __restrict__ row, int E, bool vec) {
    const int lane = lane_id();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (vec) {
            const int e = 256 * i + 4 * lane;
            const float4 f = e < E ? *reinterpret_cast<const float4*>(row + e)
                                   : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            v[i][0] = f.x; v[i][1] = f.y; v[i][2] = f.z; v[i][3] = f.w;
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int e = 256 * i + 64 * c + lane;
                v[i][c] = e < E ? row[e] : -INFINITY;
            }
        }
    }
}

// 64 neighbours a load to four a lane, and back.
template <int NV>
EM_DEV void turn_in(float (&v)[NV][4], float* lds) {
    const int lane = lane_id();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) lds[256 * i + 64 * c + lane] = v[i][c];
    wave_lds_order();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const float4 f = *reinterpret_cast<const float4*>(&lds[256 * i + 4 * lane]);
        v[i][0] = f.x; v[i][1] = f.y; v[i][2] = f.z; v[i][3] = f.w;
    }
    wave_lds_order();
}
template <int NV>
EM_DEV void store_turned(float* __restrict__ row, int E, const float (&v)[NV][4], float* lds) {
    const int lane = lane_id();
#pragma unroll
    for (int i = 0; i < NV; ++i)
        *reinterpret_cast<float4*>(&lds[256 * i + 4 * lane]) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
    wave_lds_order();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int e = 256 * i + 64 * c + lane;
            if (e < E) row[e] = lds[e];
        }
    wave_lds_order();
}

// e^v for v <= 0 from the hardware base-2 exponential: the rounding error of
// v log2(e) (up to |v| units in the last place of the result) is taken along as
// a first-order factor, which leaves that instruction's unit.  Below 2^-126: 0.
EM_DEV float exp_neg(float v) {
    constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.69314718f;
    v = v < -200.f ? -200.f : v;                        // -infinity too; NaN stays
    const float t = v * kLog2e;
    const float lo = fmaf(v, kLog2eLow, fmaf(v, kLog2e, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, lo * kLn2, e);
}

// v becomes softmax(v); the row's log sum exp is returned.  A row of -infinity
// alone (every expert masked) has no distribution: probabilities and lse 0, which
// is then the sum s; a NaN among them makes s and both NaN.
template <int NV>
EM_DEV float softmax_row(float (&v)[NV][4]) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) m = fmaxf(m, v[i][c]);
    m = wave_max(m);
    const bool none = m == -INFINITY;
    const float b = none ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            v[i][c] = exp_neg(v[i][c] - b);
            s += v[i][c];
        }
    s = wave_sum(s);
    const float inv = none ? s : 1.f / s;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) v[i][c] *= inv;
    return none ? s : m + logf(s);
}

}  // namespace

// ------------------------------------------------------------------ the load -----
// Chunk c of a.chunk tokens; its part of sequence s goes to slot c + s of the
// partial sums (both grow along the tokens, so a slot has one owner).  Bound by
// reading the logits once; they and the picks are asked for before the sequences
// are looked up.  16384 x 512: 12.8 us, 33.5 MB of logits in and 4 MB of sums out in
// one round of workgroups (2.9 TB/s: a launch and the chain of four tokens, beside
// the bytes); 333 x 64: 4.1 us, a launch and one token's chain.
template <int NV>
__global__ void __launch_bounds__(256)
rt_load(RouterLoad a) {
    __shared__ __attribute__((aligned(16))) float red[4][NV * 256];
    __shared__ int hist[NV * 256];
    __shared__ double zred[4];
    const Seqs q{a.seq_offsets, a.S, a.T};
    const int tid = threadIdx.x, lane = lane_id(), wv = wave_id();
    const int t0 = blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
    if (blockIdx.x == 0 && tid == 0) *a.done = 0;
    float row[WT][NV][4], lse[WT];                     // token t0 + wv + 4 j
#pragma unroll
    for (int j = 0; j < WT; ++j)
        if (t0 + wv + 4 * j < t1) load_row<NV>(row[j], a.logits + (int64_t)(t0 + wv + 4 * j) * a.E, a.E, a.vec);
    constexpr int PICKS = 4 * WT * 32 / 256;           // picks of a chunk per thread, at most
    int pick[PICKS];
#pragma unroll
    for (int u = 0; u < PICKS; ++u) {
        const int i = tid + 256 * u;
        pick[u] = i < (t1 - t0) * a.k ? a.topk_idx[(int64_t)t0 * a.k + i] : -1;
    }
    const int first = find_seq(q, t0);
#pragma unroll
    for (int j = 0; j < WT; ++j)
        if (t0 + wv + 4 * j < t1) {
            if (!a.vec) turn_in<NV>(row[j], red[wv]);
            lse[j] = softmax_row<NV>(row[j]);
        }
    for (int s = first; s < a.S; ++s) {
        if (q.lo(s) >= t1) break;
        const int lo = max(q.lo(s), t0), hi = min(q.hi(s), t1);
        if (lo >= hi) continue;
        for (int e = tid; e < NV * 256; e += 256) hist[e] = 0;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < PICKS; ++u) {
            const int i = tid + 256 * u;
            if ((unsigned)pick[u] < (unsigned)a.E && i >= (lo - t0) * a.k && i < (hi - t0) * a.k) atomicAdd(&hist[pick[u]], 1);
        }
        float acc[NV][4];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][c] = 0.f;
        double z2 = 0.0;
#pragma unroll
        for (int j = 0; j < WT; ++j) {
            const int t = t0 + wv + 4 * j;
            if (t < lo || t >= hi) continue;
            z2 += (double)lse[j] * (double)lse[j];
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][c] += row[j][i][c];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            *reinterpret_cast<float4*>(&red[wv][256 * i + 4 * lane]) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        if (lane == 0) zred[wv] = z2;
        __syncthreads();
        const int64_t slot = blockIdx.x + s;
        for (int e = tid; e < a.E; e += 256) {
            a.part_p[slot * a.E + e] = (red[0][e] + red[1][e]) + (red[2][e] + red[3][e]);
            a.part_c[slot * a.E + e] = hist[e];
        }
        if (tid == 0) a.part_z[slot] = (zred[0] + zred[1]) + (zred[2] + zred[3]);
        __syncthreads();
    }
}

// 64 experts of one sequence: 16 lanes rows of threads add interleaved chunks in
// float64, the rows are added in order.  The last workgroup to arrive forms the
// losses from every workgroup's dot product.  Those are passed with
// device-coherent accesses and a counted wait, not fences (a fence writes back
// the XCD's whole L2).  6.1 us at 16384 x 512, 5.2 us at 333 x 64: the launch and
// five dependent trips to memory.
__global__ void __launch_bounds__(1024)
rt_load_reduce(RouterLoad a) {
    __shared__ double sp[16][64];
    __shared__ int sc[16][64];
    __shared__ int last;
    const Seqs q{a.seq_offsets, a.S, a.T};
    const int col = threadIdx.x & 63, row = threadIdx.x >> 6;
    const int s = blockIdx.y, e = blockIdx.x * 64 + col;
    const int lo = q.lo(s), hi = q.hi(s), n = hi - lo;
    const int c0 = lo / a.chunk, c1 = n > 0 ? (hi - 1) / a.chunk + 1 : c0;
    double p = 0.0;
    int cnt = 0;
    if (e < a.E) {
#pragma unroll 4
        for (int c = c0 + row; c < c1; c += 16) {
            p += (double)a.part_p[(int64_t)(c + s) * a.E + e];
            cnt += a.part_c[(int64_t)(c + s) * a.E + e];
        }
    }
    sp[row][col] = p;
    sc[row][col] = cnt;
    __syncthreads();
    const int nblk = gridDim.x * gridDim.y;
    if (row == 0) {
        for (int r = 1; r < 16; ++r) {
            p += sp[r][col];
            cnt += sc[r][col];
        }
        const double mean = n > 0 ? p / n : 0.0;
        double dot = 0.0;
        if (e < a.E) {
            a.counts[(int64_t)s * a.E + e] = cnt;
            a.probs[(int64_t)s * a.E + e] = (float)mean;
            dot = n > 0 ? (double)cnt * mean * (double)a.E / ((double)a.k * n) : 0.0;
        }
        double z = 0.0;                                   // the sequence's z sum, by its first workgroup
        if (blockIdx.x == 0)
            for (int c = c0 + col; c < c1; c += 64) z += a.part_z[c + s];
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
            dot += __shfl_xor(dot, o, 64);
            z += __shfl_xor(z, o, 64);
        }
        if (col == 0) {
            const int id = blockIdx.y * gridDim.x + blockIdx.x;
            __hip_atomic_store(&a.dots[2 * id], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(&a.dots[2 * id + 1], z, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            last = __hip_atomic_fetch_add(a.done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (unsigned)nblk - 1;
        }
    }
    __syncthreads();
    if (!last || row != 0) return;
    double b = 0.0, z = 0.0;
    for (int i = col; i < nblk; i += 64) {
        b += __hip_atomic_load(&a.dots[2 * i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        z += __hip_atomic_load(&a.dots[2 * i + 1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        b += __shfl_xor(b, o, 64);
        z += __shfl_xor(z, o, 64);
    }
    int live, tokens;
    live_seqs(q, live, tokens);
    if (col == 0) {
        a.loss[0] = live ? (float)(b / live) : 0.f;
        a.loss[1] = tokens ? (float)(z / tokens) : 0.f;
    }
}

// ------------------------------------------------------------------ dz -----------
// One wave a token, a.chunk tokens a workgroup (each wave a run of neighbours, so
// that the sequence's f stays in registers).  The picks' terms meet the row
// through an LDS row that is zero between tokens.  Rows T .. Tp - 1 and columns
// E .. Ep - 1 of the planes are zeros.  Bound by HBM: 16384 x 512 logits in and dz
// out 16 us (67 MB, 4.2 TB/s), in and three planes out 24 to 29 us (84 MB).
template <int NV>
__global__ void __launch_bounds__(256)
rt_dlogits(RouterGrad a) {
    __shared__ __attribute__((aligned(16))) float red[4][NV * 256];
    __shared__ __attribute__((aligned(16))) float turn[4][NV * 256];
    const Seqs q{a.seq_offsets, a.S, a.T};
    const int tid = threadIdx.x, lane = lane_id(), wv = wave_id();
    const int per = a.chunk / 4;
    const int t0 = blockIdx.x * a.chunk + wv * per;
    float f[NV][4], acc[NV][4], row[WT][NV][4];
    int picks[WT];                                      // lane p has pick p, its weight and the weight's gradient
    float pw[WT], pd[WT];
#pragma unroll
    for (int j = 0; j < WT; ++j) {
        const int t = t0 + j;
        picks[j] = -1;
        pw[j] = pd[j] = 0.f;
        if (j >= per || t >= a.T) continue;
        load_row<NV>(row[j], a.logits + (int64_t)t * a.E, a.E, a.vec);
        if (a.d_topk_w && lane < a.k) {
            picks[j] = a.topk_idx[(int64_t)t * a.k + lane];
            pw[j] = a.topk_w[(int64_t)t * a.k + lane];
            pd[j] = a.d_topk_w[(int64_t)t * a.k + lane];
        }
    }
    float gb = 0.f, gz = 0.f;
    if (a.d_loss) {
        int live, tokens;
        live_seqs(q, live, tokens);
        gb = live ? a.d_loss[0] / (float)live : 0.f;
        gz = tokens ? 2.f * a.d_loss[1] / (float)tokens : 0.f;
    }
    int s = a.d_loss ? find_seq(q, t0) : 0, have = -1;
    int slo = a.d_loss ? q.lo(s) : 0, shi = a.d_loss ? q.hi(s) : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) f[i][c] = acc[i][c] = 0.f;
    float* pick_row = red[wv];                          // this wave's picks (the column sums come after them)
    if (a.d_topk_w)
#pragma unroll
        for (int i = 0; i < NV; ++i) *reinterpret_cast<float4*>(&pick_row[256 * i + 4 * lane]) = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < WT; ++j) {
        const int t = t0 + j;
        if (j >= per || t >= a.Tp) break;
        float(&d)[NV][4] = row[j];
        if (t >= a.T) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) d[i][c] = 0.f;
        } else {
            // the selection weights' gradient
            const int pick = picks[j];
            const float pv = a.d_topk_w ? pw[j] * (pd[j] - wave_sum(pw[j] * pd[j])) : 0.f;
            while (t >= shi && s + 1 < a.S) {           // the token's sequence (none: neither loss has it)
                ++s;
                slo = q.lo(s);
                shi = q.hi(s);
            }
            const bool in = a.d_loss && t >= slo && t < shi;
            if (in) {
                if (!a.vec) turn_in<NV>(d, turn[wv]);
                const float lse = softmax_row<NV>(d);
                const int n = shi - slo;
                if (have != s) {
                    have = s;
                    const float r = (float)a.E / ((float)a.k * (float)n);
#pragma unroll
                    for (int i = 0; i < NV; ++i)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int e = 256 * i + 4 * lane + c;
                            f[i][c] = e < a.E ? (float)a.counts[(int64_t)s * a.E + e] * r : 0.f;
                        }
                }
                float mean = 0.f;
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) mean = fmaf(d[i][c], f[i][c], mean);
                mean = wave_sum(mean);
                const float b = gb / (float)n, z = gz * lse;
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) d[i][c] *= fmaf(b, f[i][c] - mean, z);
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) d[i][c] = 0.f;
            }
            // an expert's picks are added in slot order by every lane that names it
            // (the order stays fixed where one is named twice), then written once
            if (a.d_topk_w) {
                float sum = 0.f;
                for (int p = 0; p < a.k; ++p) {
                    const int e = __builtin_amdgcn_readlane(pick, p);
                    const float v = __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(pv), p));
                    sum += pick == e ? v : 0.f;
                }
                const bool named = (unsigned)pick < (unsigned)a.E;
                if (named) pick_row[pick] = sum;
                wave_lds_order();
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const float4 v = *reinterpret_cast<const float4*>(&pick_row[256 * i + 4 * lane]);
                    d[i][0] += v.x; d[i][1] += v.y; d[i][2] += v.z; d[i][3] += v.w;
                }
                wave_lds_order();
                if (named) pick_row[pick] = 0.f;
                wave_lds_order();
            }
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][c] += d[i][c];
            if (a.dlogits) {
                float* out = a.dlogits + (int64_t)t * a.E;
                if (!a.vec) store_turned<NV>(out, a.E, d, turn[wv]);
                else
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int e = 256 * i + 4 * lane;
                        if (e < a.E) *reinterpret_cast<float4*>(out + e) = make_float4(d[i][0], d[i][1], d[i][2], d[i][3]);
                    }
            }
        }
        if (a.planes) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = 256 * i + 4 * lane;
                if (e >= a.Ep) continue;
                // experts past E are zero: their logits read as -infinity
                float r[4] = {d[i][0], d[i][1], d[i][2], d[i][3]};
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    const f32x2 u = {r[0], r[1]}, v = {r[2], r[3]};
                    const uint32_t a0 = __builtin_bit_cast(uint32_t, __builtin_convertvector(u, bf16x2));
                    const uint32_t a1 = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
                    *reinterpret_cast<uint2*>(a.planes + ((int64_t)p * a.Tp + t) * a.Ep + e) = make_uint2(a0, a1);
                    r[0] -= bf16_to_f32(a0 & 0xFFFFu);
                    r[1] -= bf16_to_f32(a0 >> 16);
                    r[2] -= bf16_to_f32(a1 & 0xFFFFu);
                    r[3] -= bf16_to_f32(a1 >> 16);
                }
            }
        }
    }
    if (!a.part_b) return;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        *reinterpret_cast<float4*>(&red[wv][256 * i + 4 * lane]) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    __syncthreads();
    for (int e = tid; e < a.E; e += 256)
        a.part_b[(int64_t)blockIdx.x * a.E + e] = (red[0][e] + red[1][e]) + (red[2][e] + red[3][e]);
}

// ------------------------------------------------------------------ dx, dW_r ------
// out[i][n] = sum_k A[i][k] B[k][n], A the three planes of dz and B bf16 rows:
//   DX  A = dz [t][e] (K contiguous), B = W_r;   DW  A = dz^T (K by rows), B = x
// A workgroup takes BI x 256 of out; K steps of 32 arrive by direct global -> LDS
// loads, one step ahead in two stages.  An operand whose K runs down the rows is
// transposed in registers: a lane reads a short run of columns of its eight K
// rows, and byte permutes pair the rows; operand c of lane m is then column
// 4 m + c of the run of 64, so that a lane ends with four neighbouring columns of
// out.  Three products an element, so the matrix cores bound it, with the LDS
// (16 KB a wave and step) and dx's stores close behind: waves of 64 x 64, four a
// SIMD, overlap them.  (Waves of 64 x 128, two a SIMD, read less from the LDS and
// measured the same to 5% slower, a 256-row workgroup the same.)  Both products
// and dbias share a launch: at T = 1501 neither fills the chip by itself.
// T = 16384, E = 512, d = 4096: 316 to 322 us in a long run of launches, 412 GFLOP at
// 1.3 PFLOP/s (a large library product in bf16: 1.2), the matrix cores busy 74% of the
// cycles; T = 1501: 39 to 44 us, 0.9 PFLOP/s, 448 tiles on 512 places.
// With 64 rows a SIMD has one or two waves, which then read a plane ahead of the
// products (a step 0.85 -> 0.78 us); a third and fourth LDS stage changed nothing.
namespace {

enum RtMode { RT_DX = 0, RT_DW = 1 };

template <int BI_>
struct RtCfg {
    static constexpr int BI = BI_, BN = 256, BK = 32;
    static constexpr int WN = 4, WAVES = BI / 64 * WN, TH = 64 * WAVES;   // waves of 64 rows x 64 columns
    static constexpr int NC = 4;                                     // columns a lane ends with
    static constexpr int P_B = BI * BK * 2, B_B = BK * BN * 2;       // one plane's tile, B's tile
    static constexpr int STAGE = 3 * P_B + B_B;
    static constexpr int A_INSTR = 3 * P_B / 1024 / WAVES, B_INSTR = B_B / 1024 / WAVES;
};

// Eight K rows of four bf16 columns (two words a row) to four operands of eight
// K elements.
EM_DEV void transpose8(const uint2 (&v)[8], uint4 (&o)[4]) {
    uint32_t r[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        r[i][0] = v[i].x;
        r[i][1] = v[i].y;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint32_t sel = c & 1 ? 0x07060302u : 0x05040100u;
        o[c].x = __builtin_amdgcn_perm(r[1][c / 2], r[0][c / 2], sel);
        o[c].y = __builtin_amdgcn_perm(r[3][c / 2], r[2][c / 2], sel);
        o[c].z = __builtin_amdgcn_perm(r[5][c / 2], r[4][c / 2], sel);
        o[c].w = __builtin_amdgcn_perm(r[7][c / 2], r[6][c / 2], sel);
    }
}

EM_DEV void read_rows(uint2 (&r)[8], const uint8_t* p, int row_bytes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = *reinterpret_cast<const uint2*>(p + i * row_bytes);
}

// Tiles of one product: out's row and column tiles, by slice of K.
EM_DEV int rt_row_tiles(int mode, int BI, const RouterGrad& a) { return ((mode == RT_DX ? a.T : a.E) + BI - 1) / BI; }

template <int MODE, int BI>
EM_DEV void rt_tile(const RouterGrad& a, int block, uint8_t* lds) {
    using C = RtCfg<BI>;
    constexpr int NC = C::NC;
    const int lane = lane_id(), wv = wave_id(), g = lane >> 4, m = lane & 15;
    const int wi = wv / C::WN, wn = wv % C::WN;
    const int I = MODE == RT_DX ? a.T : a.E;                 // rows of out
    const int rows_b = MODE == RT_DX ? a.E : a.T;            // rows of B
    const uint16_t* B = MODE == RT_DX ? a.w_router : a.x;
    // XCD x = block % 8 takes neighbouring tiles
    const int nn = (a.d + C::BN - 1) / C::BN, ni = rt_row_tiles(MODE, BI, a);
    const int slices = MODE == RT_DX ? a.xslices : a.slices, total = nn * ni * slices;
    const int per = (total + 7) >> 3, at = block >> 3;
    const int b = (block & 7) * per + at;
    if (at >= per || b >= total) return;
    // slices slowest (a slice's operands are shared by its tiles), then DX rows, DW columns
    const int z = slices == 1 ? 0 : b / (nn * ni), in = b - z * (nn * ni);
    const int i0 = (MODE == RT_DX ? in / nn : in % ni) * BI, n0 = (MODE == RT_DX ? in % nn : in / ni) * C::BN;
    const int K = MODE == RT_DX ? a.Ep : a.Tp;
    const int steps = K / C::BK;
    const int s0 = MODE == RT_DX && slices == 1 ? 0 : (int)((unsigned)(steps * z) / (unsigned)slices);       // steps up to 2^15
    const int s1 = MODE == RT_DX && slices == 1 ? steps : (int)((unsigned)(steps * (z + 1)) / (unsigned)slices);

    // ---- loads: 1 KB pieces of the planes' tiles, then of B's, each a uniform
    // base and a lane offset.  Tile rows and columns past the planes' (whose
    // results are not stored) read on into the workspace's spare bytes.
    const uint32_t aoff = MODE == RT_DX                      // [BI][32 e]: 64-byte rows, segments swizzled (as mx_product.hip's)
        ? (uint32_t)((lane >> 2) * a.Ep * 2 + 16 * ((lane & 3) ^ (-(lane >> 4) & 3)))
        : (uint32_t)((8 * lane / BI) * a.Ep * 2 + 2 * (8 * lane % BI));                   // [32 t][BI e]
    const uint32_t boff = 2 * min(8 * (lane & 31), a.d - 8 - n0), boff2 = boff + (lane >> 5) * a.d * 2;   // two rows a piece
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    auto fetch = [&](int st) {
        const uint32_t stage = __builtin_amdgcn_readfirstlane(base + (st & 1) * C::STAGE);
#pragma unroll
        for (int p = 0; p < C::A_INSTR; ++p) {
            const int piece = C::A_INSTR * wv + p, plane = piece / (C::P_B / 1024), in = piece % (C::P_B / 1024);
            const uint16_t* src = a.planes + (int64_t)plane * a.Tp * a.Ep
                + (MODE == RT_DX ? (int64_t)(i0 + 16 * in) * a.Ep + C::BK * st
                                 : ((int64_t)C::BK * st + 512 * in / BI) * a.Ep + i0);
            lds_load16(src, aoff, stage + 1024 * piece);
        }
#pragma unroll
        for (int p = 0; p < C::B_INSTR; ++p) {               // rows past the end repeat the last: they meet zeros
            const int piece = C::B_INSTR * wv + p, row = min(C::BK * st + 2 * piece, rows_b - 1);
            lds_load16(B + (int64_t)row * a.d + n0, row + 1 < rows_b ? boff2 : boff, stage + 3 * C::P_B + 1024 * piece);
        }
    };

    floatx4 acc[4][NC];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[i][c] = zero4();
    // A wave's LDS reads of a plane: DX the operands themselves, DW rows to transpose.
    struct Plane { uint4 v[4]; };
    auto read_plane = [&](const uint8_t* A, int p) {
        Plane o;
        if constexpr (MODE == RT_DX) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 64 * wi + 16 * i + m;
                o.v[i] = *reinterpret_cast<const uint4*>(A + p * C::P_B + r * 64 + 16 * (g ^ (-(r >> 2) & 3)));
            }
        } else {
            uint2 raw[8];
            read_rows(raw, A + p * C::P_B + 8 * g * (2 * BI) + 2 * (64 * wi + 4 * m), 2 * BI);
#pragma unroll
            for (int i = 0; i < 4; ++i) o.v[i] = make_uint4(raw[2 * i].x, raw[2 * i].y, raw[2 * i + 1].x, raw[2 * i + 1].y);
        }
        return o;
    };
    auto products = [&](const Plane& a, const uint4 (&bf)[NC]) {
        uint4 af[4];
        if constexpr (MODE == RT_DX) {
#pragma unroll
            for (int i = 0; i < 4; ++i) af[i] = a.v[i];
        } else {
            uint2 raw[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) raw[i] = i & 1 ? make_uint2(a.v[i / 2].z, a.v[i / 2].w) : make_uint2(a.v[i / 2].x, a.v[i / 2].y);
            transpose8(raw, af);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[i][c] = mfma_bf16(af[i], bf[c], acc[i][c]);
    };
    if (s0 < s1) fetch(s0);
    for (int st = s0; st < s1; ++st) {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        const uint8_t* A = lds + (st & 1) * C::STAGE;
        const uint8_t* Bt = A + 3 * C::P_B;
        const int bat = 8 * g * 512 + 2 * (16 * NC * wn + NC * m);
        uint4 bf[NC];
        uint2 raw[8];
        if constexpr (BI == 64) {
            // one or two waves a SIMD: the next plane is read, and the next step asked
            // for, under this plane's products
            read_rows(raw, Bt + bat, 512);
            const Plane p0 = read_plane(A, 0);
            if (st + 1 < s1) fetch(st + 1);
            transpose8(raw, bf);
            const Plane p1 = read_plane(A, 1);
            __builtin_amdgcn_sched_barrier(0);
            products(p0, bf);
            const Plane p2 = read_plane(A, 2);
            __builtin_amdgcn_sched_barrier(0);
            products(p1, bf);
            products(p2, bf);
        } else {
            if (st + 1 < s1) fetch(st + 1);
            read_rows(raw, Bt + bat, 512);
            transpose8(raw, bf);
#pragma unroll
            for (int p = 0; p < 3; ++p) products(read_plane(A, p), bf);
        }
    }

    // ---- out: lane holds rows of subtile i (D row 4 g + v) and columns NC m .. + NC - 1
    float* whole = MODE == RT_DX ? a.dx : a.dw_router;
    float* out = slices > 1 ? (MODE == RT_DX ? a.part_x : a.part_w) + (int64_t)z * I * a.d : whole;
    const int n = n0 + 16 * NC * wn + NC * m;
    if (n >= a.d) return;
    auto store = [&](auto past) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int r = i0 + 64 * wi + (MODE == RT_DX ? 16 * i + 4 * g + v : 4 * (4 * g + v) + i);
                if (r >= I) continue;
                float* o = out + (int64_t)r * a.d + n;
                const floatx4 w = {acc[i][0][v], acc[i][1][v], acc[i][2][v], acc[i][3][v]};
                if constexpr (decltype(past)::value) __builtin_nontemporal_store(w, reinterpret_cast<floatx4*>(o));
                else *reinterpret_cast<floatx4*>(o) = w;
            }
    };
    // a whole dx streams out past the L2, where W_r and the planes stay
    if (MODE == RT_DX && slices == 1) store(std::true_type{});
    else store(std::false_type{});
}

// 64 experts of dbias from the chunks of rt_dlogits: rows of 64 threads over
// interleaved chunks in float64, then the rows in order.
template <int TH>
EM_DEV void rt_bias(const RouterGrad& a, int block, uint8_t* lds) {
    double(*sp)[64] = reinterpret_cast<double(*)[64]>(lds);
    const int col = threadIdx.x & 63, row = threadIdx.x >> 6, e = block * 64 + col;
    const int chunks = (a.T + a.chunk - 1) / a.chunk;
    double s = 0.0;
    if (e < a.E) {
#pragma unroll 8
        for (int c = row; c < chunks; c += TH / 64) s += (double)a.part_b[(int64_t)c * a.E + e];
    }
    sp[row][col] = s;
    __syncthreads();
    if (row != 0 || e >= a.E) return;
    for (int r = 1; r < TH / 64; ++r) s += sp[r][col];
    a.dbias[e] = (float)s;
}

}  // namespace

// Workgroups: dbias (bblocks), then the tiles of dW_r (wblocks), then those of dx.
template <int BI>
__global__ void __launch_bounds__(RtCfg<BI>::TH) __attribute__((amdgpu_waves_per_eu(BI / 32)))
rt_products(RouterGrad a, int bblocks, int wblocks) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * RtCfg<BI>::STAGE];
    const int b = blockIdx.x;
    if (b < bblocks) rt_bias<RtCfg<BI>::TH>(a, b, lds);
    else if (b < bblocks + wblocks) rt_tile<RT_DW, BI>(a, b - bblocks, lds);
    else rt_tile<RT_DX, BI>(a, b - bblocks - wblocks, lds);
}

// The slices of dW_r (wblocks workgroups) and of dx, in order, eight asked for at
// once (four where there are no more): HBM and the Infinity Cache (512 x 4096, 4
// slices: 7.6 us, 42 MB).
template <int N>
EM_DEV void rt_add_slices(float4& s, const float* part, int slices, int64_t n, int64_t at, int z) {
    float4 v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = *reinterpret_cast<const float4*>(part + min(z + i, slices - 1) * n + at);
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (z + i < slices) {
            s.x += v[i].x; s.y += v[i].y; s.z += v[i].z; s.w += v[i].w;
        }
}

__global__ void __launch_bounds__(256)
rt_finish(RouterGrad a, unsigned wblocks) {
    const bool w = blockIdx.x < wblocks;
    const int64_t n = (int64_t)(w ? a.E : a.T) * a.d, at = ((int64_t)(blockIdx.x - (w ? 0 : wblocks)) * 256 + threadIdx.x) * 4;
    const float* part = w ? a.part_w : a.part_x;
    const int slices = w ? a.slices : a.xslices;
    if (at >= n) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (slices <= 4) rt_add_slices<4>(s, part, slices, n, at, 0);
    else
        for (int z = 0; z < slices; z += 8) rt_add_slices<8>(s, part, slices, n, at, z);
    *reinterpret_cast<float4*>((w ? a.dw_router : a.dx) + at) = s;
}

// ------------------------------------------------------------------ host side ----
namespace {

constexpr size_t kAl = 256;
size_t up(size_t v) { return (v + kAl - 1) & ~(kAl - 1); }

struct LoadLayout { size_t p, c, z, dots, done, bytes; };
LoadLayout load_layout(const RouterLoad& a) {
    LoadLayout L{};
    const size_t slots = (size_t)(a.T + load_chunk(a.T) - 1) / load_chunk(a.T) + a.S;
    size_t off = 0;
    auto take = [&](size_t n) { const size_t o = off; off = up(off + n); return o; };
    L.p = take(slots * a.E * 4);
    L.c = take(slots * a.E * 4);
    L.z = take(slots * 8);
    L.dots = take((size_t)a.S * ((a.E + 63) / 64) * 16);
    L.done = take(4);
    L.bytes = off;
    return L;
}

struct GradLayout { size_t planes, part_w, part_x, part_b, bytes; };

constexpr int kTileRows = 128, kPad = 32;   // largest tile of rt_products; T and E are padded to a step of K
int pad32(int v) { return (v + kPad - 1) & ~(kPad - 1); }
int64_t tiles(int rows, int bi, int d) { return (int64_t)((rows + bi - 1) / bi) * ((d + 255) / 256); }

// Tile rows of rt_products and slices of K (tokens for dW_r, experts for dx): the
// least of an estimate (us) from measured step times (32 of K).  A workgroup alone
// on a CU takes 0.85 us a step with 64 rows and 1.06 with 128, two 1.25 and 2.2
// each, and a full chip 0.85 and 1.2 us a step and CU; dx has E / 32 steps a tile,
// dW_r T / 32, split into the slices, whose sums rt_finish adds in a launch more.
// Measured passes, 64 rows against 128 (T x E x d, us): 7 x 913 x 640 30 / 40,
// 751 x 480 x 2560 30 / 33, 16384 x 512 x 4096 362 / 333; 1, 8 and 32 slices of
// 11764 x 48 x 384 282 / 52 / 30, 1, 2 and 4 of 761 x 936 x 1024 36 / 38 / 41.
void plan_grad(RouterGrad& a) {
    static constexpr double kAlone[2] = {0.85, 1.06}, kTwo[2] = {1.25, 2.2}, kFull[2] = {0.85, 1.2};
    a.Tp = pad32(a.T);
    a.Ep = pad32(a.E);
    const int tsteps = a.Tp / 32, esteps = a.Ep / 32;
    double least = 0;
    a.bi = 0;
    for (int i = 0; i < 2; ++i) {
        const int bi = 64 << i;
        const int64_t dx = tiles(a.T, bi, a.d), dw = tiles(a.E, bi, a.d);
        const double all = ((double)dx * esteps + (double)dw * tsteps) * kFull[i] / 256;
        for (int x = 1; x <= 8 && (x == 1 || 4 * x <= esteps); x *= 2)
            for (int z = 1; z <= 64 && z <= tsteps; z *= 2) {
                const int w_steps = (tsteps + z - 1) / z, x_steps = (esteps + x - 1) / x;
                const double chain = (w_steps > x_steps ? w_steps : x_steps) * (dx * x + dw * z <= 256 ? kAlone[i] : kTwo[i]);
                double finish = 0;
                if (x > 1 || z > 1)
                    finish = 3.5 + 0.3 * (z > x ? z : x) +
                             ((z > 1 ? (z + 1.0) * a.E : 0.0) + (x > 1 ? (x + 1.0) * a.T : 0.0)) * a.d * 4 / 6e6;
                const double us = (chain > all ? chain : all) + finish;
                if (!a.bi || us < least) {
                    least = us;
                    a.bi = bi;
                    a.slices = z;
                    a.xslices = x;
                }
            }
    }
}

GradLayout grad_layout(const RouterGrad& a) {
    GradLayout L{};
    size_t off = 0;
    auto take = [&](size_t n) { const size_t o = off; off = up(off + n); return o; };
    // Tiles of up to 128 rows of a T or E padded to 32: the last one reads up to 96 rows
    // past the last plane (DX), or 96 columns past its last row (DW), which is less.
    L.planes = take(((size_t)3 * a.Tp + kTileRows - kPad) * a.Ep * 2);
    L.part_w = take((size_t)(a.slices > 1 ? a.slices : 0) * a.E * a.d * 4);
    L.part_x = take((size_t)(a.xslices > 1 ? a.xslices : 0) * a.T * a.d * 4);
    L.part_b = take((size_t)((a.Tp + grad_chunk(a.T) - 1) / grad_chunk(a.T)) * a.E * 4);
    L.bytes = off;
    return L;
}

}  // namespace

size_t router_load_ws_bytes(const RouterLoad& a) { return load_layout(a).bytes; }

hipError_t launch_router_load(RouterLoad a, void* ws, hipStream_t s) {
    const LoadLayout L = load_layout(a);
    char* base = static_cast<char*>(ws);
    a.part_p = reinterpret_cast<float*>(base + L.p);
    a.part_c = reinterpret_cast<int32_t*>(base + L.c);
    a.part_z = reinterpret_cast<double*>(base + L.z);
    a.dots = reinterpret_cast<double*>(base + L.dots);
    a.done = reinterpret_cast<uint32_t*>(base + L.done);
    a.chunk = load_chunk(a.T);
    const int chunks = (a.T + a.chunk - 1) / a.chunk;
    prof_begin(s);
    if (a.E <= 256) rt_load<1><<<chunks, 256, 0, s>>>(a);
    else if (a.E <= 512) rt_load<2><<<chunks, 256, 0, s>>>(a);
    else rt_load<4><<<chunks, 256, 0, s>>>(a);
    prof_end(s, "rt_load");
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    prof_begin(s);
    rt_load_reduce<<<dim3((a.E + 63) / 64, a.S), 1024, 0, s>>>(a);
    prof_end(s, "rt_load_reduce");
    return hipGetLastError();
}

size_t router_grad_ws_bytes(RouterGrad a) {
    plan_grad(a);
    return grad_layout(a).bytes;
}

hipError_t launch_router_grad(RouterGrad a, void* ws, hipStream_t s) {
    plan_grad(a);
    const GradLayout L = grad_layout(a);
    char* base = static_cast<char*>(ws);
    a.planes = a.dx || a.dw_router ? reinterpret_cast<uint16_t*>(base + L.planes) : nullptr;
    a.part_w = reinterpret_cast<float*>(base + L.part_w);
    a.part_x = reinterpret_cast<float*>(base + L.part_x);
    a.part_b = a.dbias ? reinterpret_cast<float*>(base + L.part_b) : nullptr;
    a.chunk = grad_chunk(a.T);
    const int chunks = ((a.planes ? a.Tp : a.T) + a.chunk - 1) / a.chunk;
    prof_begin(s);
    if (a.E <= 256) rt_dlogits<1><<<chunks, 256, 0, s>>>(a);
    else if (a.E <= 512) rt_dlogits<2><<<chunks, 256, 0, s>>>(a);
    else rt_dlogits<4><<<chunks, 256, 0, s>>>(a);
    prof_end(s, "rt_dlogits");
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !(a.dx || a.dw_router || a.dbias)) return e;
    const int bi = a.bi;
    const auto up8 = [](int64_t n) { return (int)((n + 7) & ~7ll); };
    const int bblocks = a.dbias ? up8((a.E + 63) / 64) : 0;
    const int wblocks = a.dw_router ? up8(tiles(a.E, bi, a.d) * a.slices) : 0;
    const int xblocks = a.dx ? up8(tiles(a.T, bi, a.d) * a.xslices) : 0;
    prof_begin(s);
    if (bi == 128) rt_products<128><<<bblocks + wblocks + xblocks, RtCfg<128>::TH, 0, s>>>(a, bblocks, wblocks);
    else rt_products<64><<<bblocks + wblocks + xblocks, RtCfg<64>::TH, 0, s>>>(a, bblocks, wblocks);
    prof_end(s, "rt_products");
    e = hipGetLastError();
    const auto joins = [&](const float* out, int slices, int rows) {
        return out && slices > 1 ? (unsigned)(((int64_t)rows * a.d / 4 + 255) / 256) : 0u;
    };
    const unsigned wj = joins(a.dw_router, a.slices, a.E), xj = joins(a.dx, a.xslices, a.T);
    if (e != hipSuccess || !(wj + xj)) return e;
    prof_begin(s);
    rt_finish<<<wj + xj, 256, 0, s>>>(a, wj);
    prof_end(s, "rt_finish");
    return hipGetLastError();
}

}  // namespace em
