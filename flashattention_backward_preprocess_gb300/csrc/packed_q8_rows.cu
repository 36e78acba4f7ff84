// packed_q8_rows.cu -- attention over an 8-bit cache for steps of few rows (a token or a few for each
// request): packed_fwd_tc.cuh's plan, items and joins, but the numbers go from memory to registers to
// the products, with nothing in shared memory and no warp waiting for another.
//
// An item's rows (up to 16: tpt tokens x the g heads of a key/value head) are one 16-row operand of
// mma.sync m16n8k16, whose fragments a thread can load for itself.  (tcgen05 reads 128 rows of which
// such a step fills g, and takes its operands from shared memory: the 8-bit rows would have to be
// written there as fp16 first.)  Warp w of four takes keys [16 w, 16 w + 16) of each 64-key tile, with
// a max, a sum and an accumulator of its own; they meet once, at the item's end.
//   * K: the products of Q K^T run over d in an order in which a lane's operands are 16 bytes next to
//     each other: lane (q = lane / 4, t = lane % 4) loads bytes [64 x + 16 t, + 16) of keys q and q + 8.
//   * V: the output columns are numbered so that a lane needs bytes [q D / 8, + D / 8) of its four keys
//     2t, 2t + 1, 2t + 8, 2t + 9: whole 128-byte lines again; two bytes of two keys are paired by a
//     byte permutation, and pairs made fp16 by one conversion.
//   * exponents: e_k goes into the score of its key.  With y = score + e_v the weight P' = 2^(y - m)
//     stands for P 2^e_v and multiplies V's numbers as they are; the row sum takes P' 2^-e_v.  m is
//     the max of y less 8, looked at anew when a y exceeds m by 15: P' <= 2^15 fits fp16, whose fixed
//     step below 2^-14 is 2^-33 of the row's largest weight.
//   * Q is fp16, a bf16 row times a power of two (packed_q8.cuh says why).
// The next tile's loads are issued as each register is consumed; twelve warps a SM have up to 48 KB in
// flight.
#include <cuda_fp16.h>
#include <math.h>

#include "packed.cuh"
#include "packed_q8.cuh"

namespace fa {
namespace {

constexpr int RT = 16, kWarps = 4, kThreads = kWarps * 32, KT = 16 * kWarps;
constexpr int kCtas = 3;  // per SM
constexpr float kLift = 8.f, kRoom = 15.f;

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
// Byte n of a word as an exponent: 2^(b - 127), 2^(127 - b).
__device__ __forceinline__ float up2(uint32_t w, int n) { return __uint_as_float((w >> (8 * n) & 0xffu) << 23); }
__device__ __forceinline__ float down2(uint32_t w, int n) { return __uint_as_float((254u - (w >> (8 * n) & 0xffu)) << 23); }

template <typename T, int D, bool kTree>
__global__ void __launch_bounds__(kThreads, kCtas)
    q8_rows_kernel(const PackedFwd a, const FwdPlan plan, const FwdGeom geo, int max_units) {
    constexpr int X = D / 64;   // 64-column blocks of a row
    constexpr int CH = D / 8;   // V's bytes of a key per lane, output tiles of 8 columns
    constexpr int LD = D + 4;
    constexpr bool kScaleQ = TypeTraits<T>::kId == FA_BF16;
    __shared__ alignas(16) float s_o[kWarps][RT][LD];
    __shared__ uint4 s_q[X * 4][32];  // operands of Q by product step and lane
    __shared__ float2 s_ml[kWarps][RT];
    __shared__ float2 s_row[RT];
    __shared__ int s_last;
    static_assert(sizeof(SelfPlan) <= sizeof(s_o), "the plan is made where the accumulators meet later");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, q = lane >> 2, t = lane & 3;
    const int g = a.H / a.H_kv;
    ptx::griddep_wait();
    FwdShare share;
    if (geo.self) {
        SelfPlan* sp = reinterpret_cast<SelfPlan*>(&s_o[0][0][0]);
        plan_self<kThreads>(a, geo, plan, max_units, sp);
        share = sp->share;
        if (a.fill) fill_rows<T>(a, share.W == 0, blockIdx.x * kThreads + tid, (long long)gridDim.x * kThreads);
        __syncthreads();
    } else {
        share.read(plan, blockIdx.x);
    }
    const uint8_t* Kb = static_cast<const uint8_t*>(a.K);
    const uint8_t* Vb = static_cast<const uint8_t*>(a.V);
    FwdWalk w;
    for (bool more = w.init(share, blockIdx.x, a.H_kv, geo.overhead); more; more = w.next()) {
        const int rows = w.t.n_tok * g, head0 = w.hd * g;
        // ---- Q: rows q and q + 8, 16 columns of each block, as fp16 operands
        float rs[2];  // of a row: scores to log2 units
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = q + 8 * h;
            const T* Qr = static_cast<const T*>(a.Q) + (long long)(w.t.q_tok + r / g) * a.q.tok + (long long)(head0 + r % g) * a.q.head;
            uint4 raw[X][2];
            float most = 0.f;
#pragma unroll
            for (int x = 0; x < X; ++x) {
                const int c = x * 64 + t * 16;
                const bool in = r < rows && c < a.d;
                raw[x][0] = in ? reinterpret_cast<const uint4*>(Qr + c)[0] : make_uint4(0u, 0u, 0u, 0u);
                raw[x][1] = in ? reinterpret_cast<const uint4*>(Qr + c)[1] : make_uint4(0u, 0u, 0u, 0u);
            }
            int n = 0;
            if (kScaleQ) {
#pragma unroll
                for (int x = 0; x < X; ++x)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t v = (&raw[x][i >> 2].x)[i & 3];
                        const float lo = fabsf(__uint_as_float(v << 16)), hi = fabsf(__uint_as_float(v & 0xffff0000u));
                        most = fmaxf(most, fmaxf(lo <= 3.4e38f ? lo : 0.f, hi <= 3.4e38f ? hi : 0.f));
                    }
                most = quad_max(most);
                n = most > 0.f ? min(100, 14 - ((__float_as_int(most) >> 23) - 127)) : 0;
            }
            const float s = __int_as_float((n + 127) << 23);
            rs[h] = a.scale * 1.4426950408889634f * __int_as_float((127 - n) << 23);
#pragma unroll
            for (int x = 0; x < X; ++x)
#pragma unroll
                for (int i = 0; i < 8; ++i) {  // columns 2i, 2i + 1 of the lane's 16
                    uint32_t v = (&raw[x][i >> 2].x)[i & 3];
                    if (kScaleQ) v = pack_half2(__uint_as_float(v << 16) * s, __uint_as_float(v & 0xffff0000u) * s);
                    if (warp == (i >> 1)) (&s_q[x * 4 + (i >> 1)][lane].x)[(i & 1) * 2 + h] = v;
                }
        }
        __syncthreads();
        const int ctx = kTree ? w.t.pos0 - (w.t.q_tok - a.cu_q[w.t.n]) : 0;
        const int k_lo = a.window > 0 ? w.t.pos0 - a.window + 1 : 0;  // no row sees an earlier key
        const int* table = a.table + (size_t)w.t.n * a.max_pages;
        const int nt = w.tiles();
        const int first = (w.t.n_first + w.j0) * KT + warp * 16;  // this warp's first key
        // ---- loads.  A warp's 16 keys of a tile lie on one page (page_size % 16 == 0).
        auto entry_of = [&](int j) {  // table entry of the warp's keys in tile j; -2: no key there that a row sees
            const int key0 = first + j * KT;
            if (j >= nt || key0 >= w.t.S_k || key0 + 16 <= k_lo) return -2;
            const int e = key0 / a.page_size;
            return e < a.max_pages ? table[e] : -1;
        };
        uint4 kk[X][2];
        uint32_t vv[4][CH / 4];
        uint32_t ek = 0u, ev = 0u;  // exponents of keys 2t, 2t + 1, 2t + 8, 2t + 9
        auto page_at = [&](int entry) -> int {  // the page, or -1: zeros
            if (entry == -2) return -1;
            bool bad = false;
            const int pg = page_checked(entry, a.pages, &bad);
            if (bad && lane == 0) atomicOr(a.err, kErrPage);
            return bad ? -1 : pg;
        };
        auto load_k = [&](int j, int pg) {
            const int key0 = first + j * KT, in0 = key0 % a.page_size;
            const uint8_t* p = Kb + (pg < 0 ? 0 : pg * a.k_page + (long long)in0 * a.k.tok + (long long)w.hd * a.k.head) + t * 16;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int x = 0; x < X; ++x) {
                    const bool in = pg >= 0 && key0 + q + 8 * i < w.t.S_k && x * 64 + t * 16 < a.d;
                    kk[x][i] = in ? ld_once(p + (q + 8 * i) * a.k.tok + x * 64) : make_uint4(0u, 0u, 0u, 0u);
                }
            ek = ev = 0u;
            if (pg >= 0) {
                const long long e = ((long long)pg * a.H_kv + w.hd) * a.page_size + in0 + 2 * t;
                const uint16_t* pk = reinterpret_cast<const uint16_t*>(a.k_exp + e);
                const uint16_t* pv = reinterpret_cast<const uint16_t*>(a.v_exp + e);
                ek = pk[0] | (uint32_t)pk[4] << 16;
                ev = pv[0] | (uint32_t)pv[4] << 16;
            }
        };
        auto load_v = [&](int j, int pg) {
            const int key0 = first + j * KT, in0 = key0 % a.page_size;
            const uint8_t* p = Vb + (pg < 0 ? 0 : pg * a.v_page + (long long)in0 * a.v.tok + (long long)w.hd * a.v.head) + q * CH;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int r = 2 * t + (n & 1) + (n >> 1) * 8;
                const bool in = pg >= 0 && key0 + r < w.t.S_k && q * CH < a.d;
                if constexpr (CH == 16) {
                    const uint4 v = in ? ld_once(p + r * a.v.tok) : make_uint4(0u, 0u, 0u, 0u);
                    vv[n][0] = v.x, vv[n][1] = v.y, vv[n][2] = v.z, vv[n][3] = v.w;
                } else {
                    const uint2 v = in ? __ldg(reinterpret_cast<const uint2*>(p + r * a.v.tok)) : make_uint2(0u, 0u);
                    vv[n][0] = v.x, vv[n][1] = v.y;
                }
            }
        };
        float o[CH][4];
#pragma unroll
        for (int f = 0; f < CH; ++f) o[f][0] = o[f][1] = o[f][2] = o[f][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        int pg = page_at(entry_of(0));
        if (nt > 0) {
            load_k(0, pg);
            load_v(0, pg);
        }
        int next = entry_of(1);
        for (int j = 0; j < nt; ++j) {
            const int key0 = first + j * KT;
            const int after = entry_of(j + 2);
            const bool live = pg >= 0;
            // ---- scores of 16 rows and 16 keys
            float c[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.f;
#pragma unroll
            for (int x = 0; x < X; ++x)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 qw = s_q[x * 4 + k][lane];
                    const uint32_t qa[4] = {qw.x, qw.y, qw.z, qw.w};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t b0, b1;
                        e4m3x4_to_f16(k == 0 ? kk[x][i].x : k == 1 ? kk[x][i].y : k == 2 ? kk[x][i].z : kk[x][i].w, b0, b1);
                        mma_16816(c[i], qa, b0, b1);
                    }
                }
            const uint32_t ek0 = ek, ev0 = ev;
            pg = page_at(next);
            next = after;
            if (j + 1 < nt) load_k(j + 1, pg);
            // ---- weights.  c[i][2h + b]: row q + 8h, key 8i + 2t + b
            if (live) {
                const bool full = key0 + 16 <= w.t.S_k && (!a.causal || key0 + 15 <= w.t.pos0) && (!kTree || key0 + 16 <= ctx) &&
                                  (a.window <= 0 || (key0 > w.t.pos0 + w.t.n_tok - 1 - a.window &&
                                                     (a.causal || key0 + 15 < w.t.pos0 + a.window)));
                float y[2][4];
                bool grow = false;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int h = e >> 1, b = e & 1, n = 2 * i + b;
                        y[i][e] = fmaf(c[i][e], rs[h] * up2(ek0, n), (float)((int)(ev0 >> (8 * n) & 0xffu) - 127));
                        if (!full) {
                            const int key = key0 + 8 * i + 2 * t + b, r = q + 8 * h, p = w.t.pos0 + r / g;
                            bool vis = key < w.t.S_k && r < rows && key_visible(p, key, a.causal, a.window);
                            if (kTree && vis && key >= ctx) vis = tree_sees(a, w.t.q_tok + r / g, key - ctx);
                            y[i][e] = vis ? y[i][e] : -INFINITY;
                        }
                        grow |= y[i][e] > m[h] + kRoom;
                    }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float mx = quad_max(fmaxf(fmaxf(y[0][2 * h], y[0][2 * h + 1]), fmaxf(y[1][2 * h], y[1][2 * h + 1]))) - kLift;
                        if (mx > m[h]) {
                            const float alpha = m[h] == -INFINITY ? 0.f : ptx::ex2(m[h] - mx);
                            m[h] = mx;
                            l[h] *= alpha;
#pragma unroll
                            for (int f = 0; f < CH; ++f) o[f][2 * h] *= alpha, o[f][2 * h + 1] *= alpha;
                        }
                    }
                }
                const float use[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
                uint32_t pa[4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float p0 = ptx::ex2(y[i][2 * h] - use[h]), p1 = ptx::ex2(y[i][2 * h + 1] - use[h]);
                        l[h] = fmaf(p0, down2(ev0, 2 * i), fmaf(p1, down2(ev0, 2 * i + 1), l[h]));
                        pa[2 * i + h] = pack_half2(p0, p1);
                    }
                // ---- P' V
#pragma unroll
                for (int f = 0; f < CH; f += 4) {
                    const uint32_t wa = vv[0][f / 4], wb = vv[1][f / 4], wc = vv[2][f / 4], wd = vv[3][f / 4];
                    uint32_t b0, b1, b2, b3;
                    // bytes (a0, b0, a1, b1) and (a2, b2, a3, b3) of two keys' words
                    e4m3x4_to_f16(__byte_perm(wa, wb, 0x5140), b0, b2);
                    e4m3x4_to_f16(__byte_perm(wc, wd, 0x5140), b1, b3);
                    mma_16816(o[f], pa, b0, b1);
                    mma_16816(o[f + 1], pa, b2, b3);
                    e4m3x4_to_f16(__byte_perm(wa, wb, 0x7362), b0, b2);
                    e4m3x4_to_f16(__byte_perm(wc, wd, 0x7362), b1, b3);
                    mma_16816(o[f + 2], pa, b0, b1);
                    mma_16816(o[f + 3], pa, b2, b3);
                }
            }
            if (j + 1 < nt) load_v(j + 1, pg);
        }
        // ---- the four warps' parts together.  Column n of output tile f is column n CH + f of the head
        __syncthreads();  // the last item's have been read
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float sum = quad_sum(l[h]);
            if (t == 0) s_ml[warp][q + 8 * h] = make_float2(m[h], sum);
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int f = 0; f < CH; f += 4)
                    *reinterpret_cast<float4*>(&s_o[warp][q + 8 * h][(2 * t + b) * CH + f]) =
                        make_float4(o[f][2 * h + b], o[f + 1][2 * h + b], o[f + 2][2 * h + b], o[f + 3][2 * h + b]);
        }
        __syncthreads();
        const bool whole = w.whole();
        const int slot = 2 * (int)blockIdx.x + (w.j0 == 0 ? 1 : 0);
        for (int e = tid; e < rows * (D / 4); e += kThreads) {
            const int r = e / (D / 4), c4 = e % (D / 4) * 4;
            float M = -INFINITY;
#pragma unroll
            for (int v = 0; v < kWarps; ++v) M = fmaxf(M, s_ml[v][r].x);
            const float base = M == -INFINITY ? 0.f : M;
            float L = 0.f;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int v = 0; v < kWarps; ++v) {
                const float2 ml = s_ml[v][r];
                const float f = ptx::ex2(ml.x - base);
                const float4 x = *reinterpret_cast<const float4*>(&s_o[v][r][c4]);
                L = fmaf(ml.y, f, L);
                s.x = fmaf(x.x, f, s.x), s.y = fmaf(x.y, f, s.y), s.z = fmaf(x.z, f, s.z), s.w = fmaf(x.w, f, s.w);
            }
            const int tok = w.t.q_tok + r / g, head = head0 + r % g;
            if (whole) {
                if (c4 == 0) a.LSE[(size_t)head * a.T_q + tok] = lse_of(M, L);
                if (c4 >= a.d) continue;
                const float inv = inv_sum(L);
                const bool none = L == 0.f;  // 0 times a NaN in V is no 0
                alignas(8) T out[4] = {TypeTraits<T>::from_f32(none ? 0.f : s.x * inv), TypeTraits<T>::from_f32(none ? 0.f : s.y * inv),
                                       TypeTraits<T>::from_f32(none ? 0.f : s.z * inv), TypeTraits<T>::from_f32(none ? 0.f : s.w * inv)};
                *reinterpret_cast<uint2*>(static_cast<T*>(a.O) + (long long)tok * a.o.tok + (long long)head * a.o.head + c4) =
                    *reinterpret_cast<const uint2*>(out);
            } else {
                *reinterpret_cast<float4*>(plan.part_o + ((size_t)slot * RT + r) * D + c4) = s;
                if (c4 == 0) plan.part_ml[(size_t)slot * RT + r] = make_float2(part_max(M, L), L);
            }
        }
        if (!whole) {  // the last part to arrive joins the item
            int first_cta, count;
            w.parts(first_cta, count);
            __threadfence();
            __syncthreads();
            if (tid == 0) s_last = arrive_part(&plan.done[first_cta], plan.tag, count);
            __syncthreads();
            if (s_last) {
                __threadfence();
                join_parts<T, kThreads, RT, D, 2>(a, plan, w.t, head0, g, rows, first_cta, count, tid, s_row, [] { __syncthreads(); });
            }
        }
    }
}

template <typename T, int D, bool kTree>
cudaError_t launch_t(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
    const int g = a.H / a.H_kv;
    FwdGeom geo;
    geo.rows = RT;
    geo.tpt = RT / g;
    geo.bn = KT;
    geo.heads = a.H_kv;
    geo.ctas = sm_count() * kCtas;
    geo.D = D;
    geo.min_chunk = 4;
    geo.overhead = 4;  // filling the loads and the meeting of the warps
    const long long units = plan_units(a, geo);
    geo.self = units <= kSelfUnits && a.N <= kSelfUnits;
    FwdPlan plan;
    *bytes = fwd_plan_layout(a, geo, ws, &plan);
    if (ws == nullptr) return cudaSuccess;
    plan.tag = next_tag();
    cudaError_t e;
    if (!geo.self && (e = launch_fwd_plan(a, geo, plan, st)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)geo.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, q8_rows_kernel<T, D, kTree>, a, plan, geo, (int)units);
}

template <typename T>
cudaError_t launch_d(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
    if (tc_head_dim(a.d) == 64) return a.tree ? launch_t<T, 64, true>(a, ws, bytes, st) : launch_t<T, 64, false>(a, ws, bytes, st);
    return a.tree ? launch_t<T, 128, true>(a, ws, bytes, st) : launch_t<T, 128, false>(a, ws, bytes, st);
}

}  // namespace

cudaError_t launch_q8_rows(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
    return a.dtype == FA_F16 ? launch_d<__half>(a, ws, bytes, st) : launch_d<__nv_bfloat16>(a, ws, bytes, st);
}

}  // namespace fa
