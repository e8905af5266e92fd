// attn.cu -- attention over the 8-bit paged KV cache for few query rows per kv head (decode), the join of a
// split key axis, and the choice between this kernel and the tensor-memory one (attn_tc.cu).
//
// A unit is up to 16 query rows of one kv head (the rows of its group of heads, token after
// token) against a range of keys. Its four warps take 16 keys in turn, each with a running softmax
// of its own; they are joined at the end. With 16 rows the work is streaming: 2*D bytes a key,
// 64*D multiply-adds. So K and V go from memory to the registers of the thread that uses them, by
// way of a ring of private 16-byte pieces in shared memory (cp.async: 4 stages in flight
// without registers or barriers; no thread reads what another one copied), and from there as
// fp16 (exact for e4m3) into mma.m16n8k16. Both products are free to permute their contraction
// axis, so a thread's piece is 16 consecutive bytes in memory:
//   S = Q K^T: thread (r, c) = (lane / 4, lane % 4) holds key r's dims 64i + 16c .. + 15, the
//     B operand of four steps over dims; Q is laid out to match.
//   O = P V: S's accumulator is P's A operand as it stands: rows r, r + 8, keys 2c, 2c+1, 8+2c,
//     9+2c. The thread holds those four keys' dims r*D/8 .. and pairs their bytes by prmt;
//     column n of step j is dim n*D/8 + j, so a thread ends with D/4 consecutive dims of a row.
#include "attn.cuh"

namespace idx {

namespace {

constexpr int kWarps = 4;
constexpr int kStages = 4;

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// kBytes from global to this thread's piece of the ring; zeros when ok is false
template <int kBytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool ok) {
    const int n = ok ? kBytes : 0;
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(kBytes)
                     : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// One stage of a warp's ring: per lane kK 16-byte pieces of K, four kVB-byte pieces of V, scale words.
template <int D, bool kSel>
struct Ring {
    static constexpr int kK = 2 * (D / 64);
    static constexpr int kVB = D / 8;
    static constexpr int kS = kSel ? 4 : 1;  // scale words: each key's, or the block's
    static constexpr int kVAt = kK * 512, kSAt = kVAt + 4 * kVB * 32;
    static constexpr int kStage = kSAt + kS * 128;
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kLd = D + 4;  // row of the join buffer
    static constexpr int kJoin = kWarps * 16 * kLd * 4;
    static constexpr int kBytes = kRing > kJoin ? kRing : kJoin;
};

template <int D, bool kHalf, bool kSel>
__global__ void __launch_bounds__(kWarps * 32, 3) attn_rows_kernel(const AttnArgs a) {
    using R = Ring<D, kSel>;
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ float2 ml[kWarps][16];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
    pdl_wait();
    pdl_launch_dependents();

    // ---- the unit: sequence, rows, keys --------------------------------------------------------
    const int G = a.group, head = blockIdx.y, z = blockIdx.z;
    int b, row0;           // first of the unit's rows: (token of the sequence) * G + head of the group
    int64_t tok0;          // query row that row 0 counts from
    int rows, kv_end;      // rows that exist; end of the keys (entries) that some row may see
    SeqRows s;
    if constexpr (kSel) {
        const int tiles = (G + 15) / 16;
        const int64_t t = blockIdx.x / tiles;
        b = seq_of_query(a.cu_seqlens_q, a.B, t);
        if (b < 0) return;
        s = seq_rows(a, b);
        row0 = (int)(blockIdx.x % tiles) * 16;
        tok0 = t;
        rows = min(16, G - row0);
        kv_end = a.n_sel;
    } else {
        const int tiles = (int)(((int64_t)a.max_q_len * G + 15) / 16);
        b = blockIdx.x / tiles;
        s = seq_rows(a, b);
        row0 = (int)(blockIdx.x % tiles) * 16;
        tok0 = s.t0;
        rows = min((int64_t)16, (int64_t)s.nq * G - row0);
        kv_end = 0;
    }
    if (s.nq < 0) {
        if (tid == 0 && head == 0 && z == 0) report(a.dev_status, IDX_STATUS_BAD_LEN);
        return;
    }
    if (rows <= 0) return;
    int vis[2];  // keys that rows r and r + 8 see
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = row0 + min(r + 8 * i, rows - 1);
        const int64_t tok = kSel ? tok0 - s.t0 : row / G;
        vis[i] = (int)visible_keys(s.len, s.nq, tok, a.causal);
    }
    if constexpr (!kSel) kv_end = (int)visible_keys(s.len, s.nq, (row0 + rows - 1) / G, a.causal);
    const int k0 = z * a.chunk, k1 = min(kv_end, k0 + a.chunk);

    // ---- q: fp16, laid out for the contraction over a thread's 16 consecutive dims ----------------
    uint32_t qa[D / 64][4][4];
    float rc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = row0 + min(r + 8 * i, rows - 1);
        const int64_t tok = kSel ? tok0 : tok0 + row / G;
        const uint16_t* q = a.q + tok * a.q_row_stride + (int64_t)(head * G + (kSel ? row : row % G)) * a.q_head_stride;
        uint4 w[D / 64][2];
        float amax = 0.0f;
        bool odd = false;  // an infinity or a NaN
#pragma unroll
        for (int d = 0; d < D / 64; ++d)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w[d][h] = *reinterpret_cast<const uint4*>(q + 64 * d + 16 * c + 8 * h);
                const uint32_t* u = reinterpret_cast<const uint32_t*>(&w[d][h]);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float2 f = load_pair<kHalf>(u[x]);
                    odd |= !(fabsf(f.x) < __int_as_float(0x7f800000)) || !(fabsf(f.y) < __int_as_float(0x7f800000));
                    amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
            odd |= __shfl_xor_sync(kFull, (int)odd, o) != 0;
        }
        const int e = odd ? 0 : q_exponent<kHalf>(amax);
        const float up = pow2f(-e);
        rc[i] = odd ? __int_as_float(0x7fc00000) : a.scale * kLog2e * pow2f(e);
#pragma unroll
        for (int d = 0; d < D / 64; ++d)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t* u = reinterpret_cast<const uint32_t*>(&w[d][h]);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t v = u[x];
                    if constexpr (!kHalf) {
                        const float2 f = load_pair<kHalf>(v);
                        v = half2_bits(f.x * up, f.y * up);
                    }
                    // word x of half h: dims 8h + 2x, + 1 of the 16: step 2h + x/2, first or second pair
                    qa[d][2 * h + x / 2][2 * (x & 1) + i] = v;
                }
            }
    }

    // ---- the key loop -------------------------------------------------------------------------------
    uint8_t* ring = sm + warp * kStages * R::kStage;
    const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + 16 * lane;
    const uint32_t ring_v = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + R::kVAt + R::kVB * lane;
    const uint32_t ring_x = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + R::kSAt + 4 * lane;
    const int P = a.page_size, lp = P == 128 ? 7 : 6;
    const int64_t hb = kv_head_bytes(P, D);
    const uint8_t* pool = a.pool + (int64_t)head * hb;
    const int32_t* pt = a.page_table + (int64_t)b * a.pt_stride;
    const int n_it = k1 > k0 ? (k1 - k0 - 16 * warp + 16 * kWarps - 1) / (16 * kWarps) : 0;
    const int kw = k0 + 16 * warp;  // this warp's first key; its next ones are 16 * kWarps further
    bool bad_page = false;

    // Lookups run ahead of the copies: the page of step it + 1 (and, with a list, the entry of
    // step it + 2) is loaded while step it's copies are issued. With a list, lane l holds entry l.
    int32_t page_n = -1, entry_n = -1, entry_c = -1;
    auto load_entry = [&](int it) -> int32_t {
        const int e = kw + 16 * kWarps * it + (lane & 15);
        return (it < n_it && e < k1) ? a.sel[tok0 * a.sel_stride + e] : -1;
    };
    auto load_page = [&](int it, int32_t entry) -> int32_t {
        if constexpr (kSel) {
            return (entry >= 0 && entry < vis[0]) ? pt[entry >> lp] : -1;
        } else {
            return it < n_it ? pt[(kw + 16 * kWarps * it) >> lp] : -1;
        }
    };
    uint32_t valid = 0;  // 4 bits per stage: the thread's keys 2c, 2c+1, 8+2c, 9+2c may be used
    uint32_t half_sel = 0;  // 4 bits per stage: which half of the scale word is the key's (list)
    auto issue = [&](int it) {
        const int st = it & (kStages - 1);
        const uint32_t at = st * R::kStage;
        if constexpr (kSel) {
            int32_t page = page_n;
            const int32_t ent = entry_c;
            const bool seen = it < n_it && ent >= 0 && ent < vis[0];
            if (seen && (uint32_t)page >= (uint64_t)a.num_pages) bad_page = true;
            if (!seen || (uint32_t)page >= (uint64_t)a.num_pages) page = -1;
            const int32_t tok = ent & (P - 1);
            valid &= ~(15u << (4 * st));
            half_sel &= ~(15u << (4 * st));
#pragma unroll
            for (int j = 0; j < 2; ++j) {  // K: keys r, 8 + r
                const int32_t pg = __shfl_sync(kFull, page, 8 * j + r), tk = __shfl_sync(kFull, tok, 8 * j + r);
                const uint8_t* src = pool + (pg < 0 ? 0 : (int64_t)pg * a.page_stride + (int64_t)tk * 2 * D) + 16 * c;
#pragma unroll
                for (int d = 0; d < D / 64; ++d)
                    cp_async<16>(ring_s + at + (j * (D / 64) + d) * 512, src + 64 * d, pg >= 0);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // V and scales: keys 2c, 2c+1, 8+2c, 9+2c
                const int from = (k >> 1) * 8 + 2 * c + (k & 1);
                const int32_t pg = __shfl_sync(kFull, page, from), tk = __shfl_sync(kFull, tok, from);
                const uint8_t* base = pool + (pg < 0 ? 0 : (int64_t)pg * a.page_stride);
                const int t2 = pg < 0 ? 0 : tk;
                cp_async<R::kVB>(ring_v + at + k * R::kVB * 32, base + (int64_t)t2 * 2 * D + D + r * R::kVB, pg >= 0);
                cp_async<4>(ring_x + at + k * 128, base + 2ll * P * D + ((t2 / kKvBlock) & ~1) * 2, pg >= 0);
                valid |= (pg >= 0 ? 1u : 0u) << (4 * st + k);
                half_sel |= ((t2 / kKvBlock) & 1u) << (4 * st + k);
            }
        } else {
            const int kb = kw + 16 * kWarps * it;
            const bool in = it < n_it;
            const bool okp = in && (uint32_t)page_n < (uint64_t)a.num_pages;
            if (in && !okp) bad_page = true;
            const int tk = kb & (P - 1);
            const uint8_t* base = pool + (okp ? (int64_t)page_n * a.page_stride : 0);
            const uint8_t* tok = base + (okp ? (int64_t)tk * 2 * D : 0);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int d = 0; d < D / 64; ++d)
                    cp_async<16>(ring_s + at + (j * (D / 64) + d) * 512,
                                 tok + (8 * j + r) * 2 * D + 16 * c + 64 * d, okp && kb + 8 * j + r < k1);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int key = (k >> 1) * 8 + 2 * c + (k & 1);
                cp_async<R::kVB>(ring_v + at + k * R::kVB * 32, tok + key * 2 * D + D + r * R::kVB,
                                 okp && kb + key < k1);
            }
            cp_async<4>(ring_x + at, base + 2ll * P * D + (okp ? ((tk / kKvBlock) & ~1) * 2 : 0), okp);
            valid = (valid & ~(1u << st)) | (okp ? 1u : 0u) << st;
        }
        cp_async_commit();
    };

    float m[2] = {neg_inf(), neg_inf()}, l[2] = {0.0f, 0.0f};
    float o[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[j][x] = 0.0f;

    if (n_it > 0) {
        entry_c = kSel ? load_entry(0) : -1;
        entry_n = kSel ? load_entry(1) : -1;
        page_n = load_page(0, entry_c);
#pragma unroll 1
        for (int it = -(kStages - 1); it < n_it; ++it) {
            const int ahead = it + kStages - 1;
            {
                const int32_t e2 = kSel ? load_entry(ahead + 2) : -1;
                const int32_t p2 = load_page(ahead + 1, entry_n);
                issue(ahead);
                page_n = p2;
                entry_c = entry_n;
                entry_n = e2;
            }
            if (it < 0) continue;
            cp_async_wait<kStages - 1>();
            const int st = it & (kStages - 1);
            const uint8_t* sp = ring + st * R::kStage;

            float sc[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int x = 0; x < 4; ++x) sc[j][x] = 0.0f;
#pragma unroll
                for (int d = 0; d < D / 64; ++d) {
                    const uint4 w = *reinterpret_cast<const uint4*>(sp + (j * (D / 64) + d) * 512 + 16 * lane);
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        uint32_t lo, hi;
                        e4m3x4_to_f16x4(u[x], lo, hi);
                        mma16816(sc[j], qa[d][x], lo, hi);
                    }
                }
            }
            // u = s * c + Ev for the thread's four keys and two rows; masked ones to -inf
            float ev[4], kc[4];
            const int kb = kw + 16 * kWarps * it;
            if constexpr (kSel) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(sp + R::kSAt + k * 128 + 4 * lane);
                    const uint32_t by = (half_sel >> (4 * st + k)) & 1u ? w >> 16 : w;
                    kc[k] = k_scale(by);
                    ev[k] = v_exponent(by);
                }
            } else {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(sp + R::kSAt + 4 * lane);
                const uint32_t by = ((kb & (P - 1)) / kKvBlock) & 1 ? w >> 16 : w;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    kc[k] = k_scale(by);
                    ev[k] = v_exponent(by);
                }
            }
            float mx[2] = {neg_inf(), neg_inf()};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float& v = sc[k >> 1][2 * i + (k & 1)];
                    bool see;
                    if constexpr (kSel)
                        see = (valid >> (4 * st + k)) & 1u;
                    else
                        see = ((valid >> st) & 1u) && kb + 8 * (k >> 1) + 2 * c + (k & 1) < vis[i];
                    v = see ? fmaf(v, rc[i] * kc[k], ev[k]) : neg_inf();
                    mx[i] = fmaxf(mx[i], v);
                }
            }
            bool raise = false;
            float f[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(kFull, mx[i], 1));
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(kFull, mx[i], 2));
                f[i] = 1.0f;
                if (mx[i] > m[i] + kLazy) {  // from -inf too
                    f[i] = ex2(m[i] - mx[i]);
                    m[i] = mx[i];
                    raise = true;
                }
            }
            if (__any_sync(kFull, raise)) {
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    o[j][0] *= f[0]; o[j][1] *= f[0];
                    o[j][2] *= f[1]; o[j][3] *= f[1];
                }
                l[0] *= f[0];
                l[1] *= f[1];
            }
            uint32_t pa[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // a row that saw nothing yet: its weights are 2^-inf
                const float sub = m[i] == neg_inf() ? 0.0f : kShift - m[i];
                float p[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) p[k] = ex2(sc[k >> 1][2 * i + (k & 1)] + sub);
                if constexpr (kSel) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        l[i] = fmaf(p[k], (valid >> (4 * st + k)) & 1u ? ex2(-ev[k]) : 0.0f, l[i]);
                } else {
                    l[i] = fmaf(p[0] + p[1] + p[2] + p[3], (valid >> st) & 1u ? ex2(-ev[0]) : 0.0f, l[i]);
                }
                pa[i] = half2_bits(p[0], p[1]);
                pa[2 + i] = half2_bits(p[2], p[3]);
            }
            // O += P V
#pragma unroll
            for (int h = 0; h < (D == 128 ? 2 : 1); ++h) {  // 8 dims at a time
                uint2 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = *reinterpret_cast<const uint2*>(sp + R::kVAt + k * R::kVB * 32 + R::kVB * lane + 8 * h);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t w0 = x ? v[0].y : v[0].x, w1 = x ? v[1].y : v[1].x;
                    const uint32_t w2 = x ? v[2].y : v[2].x, w3 = x ? v[3].y : v[3].x;
                    uint32_t b0[4], b1[4];
                    e4m3x4_to_f16x4(__byte_perm(w0, w1, 0x5140), b0[0], b0[1]);
                    e4m3x4_to_f16x4(__byte_perm(w0, w1, 0x7362), b0[2], b0[3]);
                    e4m3x4_to_f16x4(__byte_perm(w2, w3, 0x5140), b1[0], b1[1]);
                    e4m3x4_to_f16x4(__byte_perm(w2, w3, 0x7362), b1[2], b1[3]);
#pragma unroll
                    for (int y = 0; y < 4; ++y) mma16816(o[8 * h + 4 * x + y], pa, b0[y], b1[y]);
                }
            }
        }
        cp_async_wait<0>();
    }
    if (bad_page) report(a.dev_status, IDX_STATUS_BAD_PAGE);

    // ---- join the warps ------------------------------------------------------------------------------
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(kFull, l[i], 1);
        l[i] += __shfl_xor_sync(kFull, l[i], 2);
    }
    __syncthreads();  // every warp is done with its ring
    float* join = reinterpret_cast<float*>(sm);
    if (c == 0) {
        ml[warp][r] = make_float2(m[0], l[0]);
        ml[warp][r + 8] = make_float2(m[1], l[1]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float* dst = join + (warp * 16 + r + 8 * i) * R::kLd + 2 * c * (D / 8);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int j = 0; j < D / 8; j += 4)
                *reinterpret_cast<float4*>(dst + x * (D / 8) + j) =
                    make_float4(o[j][2 * i + x], o[j + 1][2 * i + x], o[j + 2][2 * i + x], o[j + 3][2 * i + x]);
    }
    __syncthreads();
    for (int e = tid; e < 16 * (D / 4); e += kWarps * 32) {
        const int row = e / (D / 4), d4 = e % (D / 4);
        if (row >= rows) continue;
        float M = neg_inf();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w][row].x);
        float L = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float2 x = ml[w][row];
            const float g = x.x == M ? 1.0f : ex2(x.x - M);
            const float4 y = *reinterpret_cast<const float4*>(join + (w * 16 + row) * R::kLd + 4 * d4);
            L = fmaf(g, x.y, L);
            v.x = fmaf(g, y.x, v.x); v.y = fmaf(g, y.y, v.y);
            v.z = fmaf(g, y.z, v.z); v.w = fmaf(g, y.w, v.w);
        }
        const int at = row0 + row;
        const int64_t tok = kSel ? tok0 : tok0 + at / G;
        const int hq = head * G + (kSel ? at : at % G);
        if (a.n_split > 1) {
            const int64_t pr = ((int64_t)z * a.T + tok) * a.q_heads + hq;
            if (!(L == 0.0f)) *reinterpret_cast<float4*>(a.part_o + pr * D + 4 * d4) = v;
            if (d4 == 0) a.part_ml[pr] = make_float2(M, L);
        } else {
            const float g = L == 0.0f ? 0.0f : 1.0f / L;
            uint2 w;
            w.x = store_pair<kHalf>(v.x * g, v.y * g);
            w.y = store_pair<kHalf>(v.z * g, v.w * g);
            *reinterpret_cast<uint2*>(a.out + tok * a.out_row_stride + (int64_t)hq * a.out_head_stride + 4 * d4) = w;
            if (a.lse && d4 == 0) a.lse[tok * a.q_heads + hq] = lse_of(M, L);
        }
    }
}

// Joins the splits of a key axis: a warp per (query row, head).
template <int D, bool kHalf>
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnArgs a) {
    constexpr int kPer = D / 32;  // dims of a lane
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if (row >= a.T * a.q_heads) return;
    const int64_t t = row / a.q_heads;
    const int hq = (int)(row % a.q_heads);
    const int b = seq_of_query(a.cu_seqlens_q, a.B, t);
    if (b < 0 || seq_rows(a, b).nq < 0) return;
    const int64_t step = a.T * a.q_heads;
    float M = neg_inf();
    for (int z = lane; z < a.n_split; z += 32) M = fmaxf(M, a.part_ml[row + z * step].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    float L = 0.0f, v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = 0.0f;
#pragma unroll 4
    for (int z = 0; z < a.n_split; ++z) {
        const int64_t pr = row + z * step;
        const float2 x = a.part_ml[pr];
        if (x.y == 0.0f) continue;  // that split had no key for this row and wrote no O
        const float g = x.x == M ? 1.0f : ex2(x.x - M);
        L = fmaf(g, x.y, L);
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = fmaf(g, a.part_o[pr * D + kPer * lane + i], v[i]);
    }
    const float g = L == 0.0f ? 0.0f : 1.0f / L;
    uint32_t* out = reinterpret_cast<uint32_t*>(a.out + t * a.out_row_stride + (int64_t)hq * a.out_head_stride + kPer * lane);
#pragma unroll
    for (int i = 0; i < kPer; i += 2) out[i / 2] = store_pair<kHalf>(v[i] * g, v[i + 1] * g);
    if (a.lse && lane == 0) a.lse[row] = lse_of(M, L);
}

// Rows that share their keys: those of a sequence and a kv head, or with a list those of a query's group.
int64_t shared_rows(const AttnArgs& a) { return a.n_sel ? a.group : (int64_t)a.max_q_len * a.group; }
// More rows than one mma.sync tile: the tensor-memory kernel.
bool use_tile(const AttnArgs& a) { return shared_rows(a) > 16; }

template <int D, bool kHalf, bool kSel>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t st) {
    constexpr int smem = Ring<D, kSel>::kBytes;
    auto* kernel = attn_rows_kernel<D, kHalf, kSel>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(allowed, kernel, smem);
    if (e != cudaSuccess) return e;
    const int64_t units = kSel ? a.T * ((a.group + 15) / 16)
                               : a.B * (((int64_t)a.max_q_len * a.group + 15) / 16);
    return launch_pdl(kernel, dim3((unsigned)units, (unsigned)a.kv_heads, (unsigned)a.n_split), dim3(kWarps * 32), smem,
                      st, a);
}

template <int D, bool kHalf>
cudaError_t launch_d(const AttnArgs& a, cudaStream_t st) {
    cudaError_t e = use_tile(a) ? launch_attn_tile(a, st)
                    : a.sel     ? launch_rows<D, kHalf, true>(a, st)
                                : launch_rows<D, kHalf, false>(a, st);
    if (e != cudaSuccess || a.n_split <= 1) return e;
    const int64_t rows = a.T * a.q_heads;
    return launch_pdl(attn_join_kernel<D, kHalf>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, st, a);
}

}  // namespace

int64_t attn_plan(AttnArgs& a, int64_t bytes) {
    const int sms = device_sm_count();
    if (sms <= 0) return -1;
    const bool tile = use_tile(a);
    const int64_t per_unit = tile ? 128 : 16;
    const int64_t units = (a.n_sel ? a.T : a.B) * ((shared_rows(a) + per_unit - 1) / per_unit) * a.kv_heads;
    const int64_t keys = a.n_sel ? a.n_sel : a.max_seq_len_k;
    const int64_t per_split = a.T * a.q_heads * (a.head_dim + 2) * 4;
    // two rounds of resident CTAs (three or two to an SM), four steps of keys to a CTA at least
    const int64_t slots = 2ll * sms * (tile ? 2 : 3), least = tile ? 512 : 256;
    int64_t want = units > 0 ? (slots + units - 1) / units : 1;
    want = want < (keys + least - 1) / least ? want : (keys + least - 1) / least;
    want = want > 64 ? 64 : want;
    if (want < 1) want = 1;
    const int64_t fits = per_split > 0 ? bytes / per_split : 1;
    int64_t n = want < fits ? want : fits;
    if (n < 1) n = 1;
    int64_t chunk = ((keys + n - 1) / n + 127) / 128 * 128;  // whole steps and pages
    if (chunk < 128) chunk = 128;
    n = (keys + chunk - 1) / chunk;
    if (n < 1) n = 1;
    a.n_split = (int32_t)n;
    a.chunk = (int32_t)chunk;
    return want > 1 ? want * per_split : 0;
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t st) {
    if (a.head_dim == 128) return a.ftype == IDX_FP16 ? launch_d<128, true>(a, st) : launch_d<128, false>(a, st);
    return a.ftype == IDX_FP16 ? launch_d<64, true>(a, st) : launch_d<64, false>(a, st);
}

}  // namespace idx
