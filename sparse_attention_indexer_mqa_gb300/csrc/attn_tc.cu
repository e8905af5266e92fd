// attn_tc.cu -- attention over the 8-bit paged KV cache for many query rows per kv head (prefill, chunks,
// large groups of heads) on the tensor cores with tensor-memory accumulators.
//
// A unit is a tile of 128 query rows of one kv head (token-major: row = token * group + head of the
// group; with a list of keys, the group's heads of one token) against a range of keys, 128 at a
// time: S = Q K^T (M = 128 rows, N = 128 keys), the running softmax of attn.cuh, O += P V (N = D). S and
// O live in tensor memory (128 + D columns), P overwrites S as fp16 and is the second product's A
// operand from there. Roles of a CTA's eight warps:
//   0-3  softmax: thread = row. Q to shared memory at the start, S -> P per tile, O out at the end;
//   4-7  converters: e4m3 from memory to fp16 operand tiles in shared memory (exact). The loads of
//        a tile go out one tile ahead into registers, so any row order costs the same: pages
//        and lists of keys need no gather pass. V is transposed on the way (8 keys x 16 dims per
//        thread, bytes paired by prmt), which makes both products K-major;
//   7    one of its threads issues the MMAs between its own conversions (a ninth warp would cost
//        every thread a quarter of its registers).
// fp16 runs at half the 8-bit rate, but 8-bit operands would leave q and the weights 4 bits; two
// 8-bit halves each would cost the same tensor time and more conversion. Two CTAs share an SM
// (tensor memory 2 x 256 columns, shared memory 2 x 103 KB): one's products run under the other's
// softmax.
#include "attn.cuh"
#include "tc.cuh"

namespace idx {

namespace {

constexpr int kRowsT = 128;   // rows of a tile
constexpr int kKeysT = 128;   // keys of a step
constexpr int kThreadsT = 256;

template <int D>
struct SmemT {
    static constexpr int kQ = 0;                            // [D/64][128 rows][128 B]
    static constexpr int kK = kQ + kRowsT * D * 2;          // [D/64][128 keys][128 B]
    static constexpr int kV = kK + kKeysT * D * 2;          // [2][D dims][128 B]
    static constexpr int kScale = kV + kKeysT * D * 2;      // [2][128] float4: 2^Ek, Ev, 2^-Ev
    static constexpr int kOff = kScale + 2 * kKeysT * 16;   // [2][128] int64: a listed key's row in the pool
    static constexpr int kBar = kOff + 2 * kKeysT * 8;
    static constexpr int kBytes = kBar + 64 + 1024;         // 1024: alignment of the operand tiles
};

// Barriers of the four converter warps, one of them with a vote.
__device__ __forceinline__ void conv_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool conv_all(bool v) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}
// Bounded wait of a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(kFull, tc::mbar_wait(bar, parity));
}

template <int D, bool kHalf, bool kSel>
__global__ void __launch_bounds__(kThreadsT, 2) attn_tile_kernel(const AttnArgs a) {
    using S = SmemT<D>;
    extern __shared__ uint8_t sm_raw[];
    __shared__ uint32_t tmem_slot;
    uint8_t* sm = sm_raw + ((1024u - (tc::smem_u32(sm_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::kBar);
    uint64_t *q_full = bars, *k_full = bars + 1, *v_full = bars + 2, *s_full = bars + 3, *p_full = bars + 4,
             *o_done = bars + 5, *drain = bars + 6;
    float4* scales = reinterpret_cast<float4*>(sm + S::kScale);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        tc::mbar_init(q_full, kRowsT);
        tc::mbar_init(k_full, 128);
        tc::mbar_init(v_full, 128);
        tc::mbar_init(s_full, 1);
        tc::mbar_init(p_full, kRowsT);
        tc::mbar_init(o_done, 1);
        tc::mbar_init(drain, 1);
        tc::fence_mbar_init();
    }
    pdl_wait();

    // ---- the unit ------------------------------------------------------------------------------
    const int G = a.group, head = blockIdx.y, z = blockIdx.z;
    int b, row0, rows, kv_end = 0;
    int64_t tok0;
    SeqRows s;
    if constexpr (kSel) {
        const int tiles = (G + kRowsT - 1) / kRowsT;
        const int64_t t = blockIdx.x / tiles;
        b = seq_of_query(a.cu_seqlens_q, a.B, t);
        if (b >= 0) s = seq_rows(a, b);
        row0 = (int)(blockIdx.x % tiles) * kRowsT;
        tok0 = t;
        rows = b < 0 ? 0 : min(kRowsT, G - row0);
        kv_end = a.n_sel;
    } else {
        // the last rows of a sequence see the most keys and go first
        const int tiles = (int)(((int64_t)a.max_q_len * G + kRowsT - 1) / kRowsT);
        b = blockIdx.x % a.B;
        s = seq_rows(a, b);
        row0 = (tiles - 1 - (int)(blockIdx.x / a.B)) * kRowsT;
        tok0 = s.t0;
        rows = (int)max((int64_t)0, min((int64_t)kRowsT, (int64_t)s.nq * G - row0));
        if (rows > 0) kv_end = (int)visible_keys(s.len, s.nq, (row0 + rows - 1) / G, a.causal);
    }
    if (b >= 0 && s.nq < 0) {
        if (tid == 0 && head == 0 && z == 0) report(a.dev_status, IDX_STATUS_BAD_LEN);
        rows = 0;
    }
    // uniform: nothing has been allocated yet
    if (rows <= 0) {
        pdl_launch_dependents();
        return;
    }
    if (warp == 7) {
        tc::tmem_alloc(&tmem_slot, 256);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    pdl_launch_dependents();  // with the tensor memory in hand: a dependent may allocate its own
    const uint32_t tm_s = tmem_slot, tm_o = tm_s + 128;
    const int k0 = z * a.chunk, k1 = min(kv_end, k0 + a.chunk);
    const int n = k1 > k0 ? (k1 - k0 + kKeysT - 1) / kKeysT : 0;
    bool ok = true;

    if (warp < 4) {
        // ---- softmax: this thread's row --------------------------------------------------------------
        const bool real = tid < rows;
        const int row = row0 + min(tid, rows - 1);
        const int64_t tok = kSel ? tok0 : tok0 + row / G;
        const int hq = head * G + (kSel ? row : row % G);
        const int vis = (int)visible_keys(s.len, s.nq, tok - s.t0, a.causal);
        float rc = 0.0f;
        {
            const uint4* q = reinterpret_cast<const uint4*>(a.q + tok * a.q_row_stride + (int64_t)hq * a.q_head_stride);
            uint4 w[D / 8];
            float amax = 0.0f;
            bool odd = false;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                w[i] = real ? q[i] : make_uint4(0, 0, 0, 0);
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float2 f = load_pair<kHalf>(u[x]);
                    odd |= !(fabsf(f.x) < __int_as_float(0x7f800000)) || !(fabsf(f.y) < __int_as_float(0x7f800000));
                    amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
            const int e = odd ? 0 : q_exponent<kHalf>(amax);
            const float up = pow2f(-e);
            rc = odd ? __int_as_float(0x7fc00000) : a.scale * kLog2e * pow2f(e);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                if constexpr (!kHalf) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float2 f = load_pair<kHalf>(u[x]);
                        u[x] = half2_bits(f.x * up, f.y * up);
                    }
                }
                *reinterpret_cast<uint4*>(sm + S::kQ + (i / 8) * (kRowsT * 128) + tid * 128 +
                                          (((i & 7) ^ (tid & 7)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
            }
            tc::fence_proxy_async();
            tc::mbar_arrive(q_full);
        }
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const bool idle = 32 * warp >= rows;  // no row of this warp exists
        float m = neg_inf(), l = 0.0f;
        for (int j = 0; j < n && ok; ++j) {
            ok = warp_wait(s_full, j & 1);
            if (!ok) break;
            if (!idle) {
                tc::tc_fence_after();
                const float4* sc = scales + (j & 1) * kKeysT;
                const int kt = k0 + j * kKeysT;
                const bool cut = !kSel && __any_sync(kFull, kt + kKeysT > vis);
                float mx = neg_inf();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t r[32];
                    __syncwarp();
                    tc::tmem_ld32(tm_s + lanes + 32 * c, r);
                    tc::tmem_ld_wait();
                    if constexpr (kSel) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float4 k = sc[32 * c + i];
                            mx = fmaxf(mx, fmaf(__uint_as_float(r[i]), rc * k.x, k.y));
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float4 k = sc[2 * c + h];
                            float bm = neg_inf();
                            if (cut) {
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    if (kt + 32 * c + 16 * h + i < vis) bm = fmaxf(bm, __uint_as_float(r[16 * h + i]));
                            } else {
#pragma unroll
                                for (int i = 0; i < 16; ++i) bm = fmaxf(bm, __uint_as_float(r[16 * h + i]));
                            }
                            // nothing visible: bm is -inf, and so is the sum whatever the factor's sign of zero
                            if (bm > neg_inf()) mx = fmaxf(mx, fmaf(bm, rc * k.x, k.y));
                        }
                    }
                }
                float f = 1.0f;
                const bool raise = mx > m + kLazy;
                if (raise) {
                    f = ex2(m - mx);
                    m = mx;
                    l *= f;
                }
                if (j > 0 && __any_sync(kFull, raise)) {
                    // s_full is committed behind the previous O += P V, so O is complete
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t r[16];
                        __syncwarp();
                        tc::tmem_ld16(tm_o + lanes + 16 * c, r);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
                        tc::tmem_st16(tm_o + lanes + 16 * c, r);
                    }
                }
                const float top = m == neg_inf() ? 0.0f : kShift - m;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t r[32], p2[16];
                    __syncwarp();
                    tc::tmem_ld32(tm_s + lanes + 32 * c, r);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float cc = 0.0f, sub = 0.0f, inv = 0.0f, sum = 0.0f;
                        if constexpr (!kSel) {
                            const float4 k = sc[2 * c + h];
                            cc = rc * k.x;
                            sub = k.y + top;
                            inv = k.z;
                        }
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            float p[2];
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const int at = 16 * h + i + y;
                                if constexpr (kSel) {
                                    const float4 k = sc[32 * c + at];
                                    p[y] = ex2(fmaf(__uint_as_float(r[at]), rc * k.x, k.y + top));
                                    l = fmaf(p[y], k.z, l);
                                } else {
                                    float u = fmaf(__uint_as_float(r[at]), cc, sub);
                                    if (cut) u = kt + 32 * c + at < vis ? u : neg_inf();
                                    p[y] = ex2(u);
                                    sum += p[y];
                                }
                            }
                            p2[8 * h + i / 2] = half2_bits(p[0], p[1]);
                        }
                        if constexpr (!kSel) l = fmaf(sum, inv, l);
                    }
                    // columns 16c .. 16c+15 held scores that were read in step c or before
                    tc::tmem_st16(tm_s + lanes + 16 * c, p2);
                }
                tc::tmem_st_wait();
                tc::tc_fence_before();
            }
            tc::mbar_arrive(p_full);
        }
        // ---- the row's result -------------------------------------------------------------------------
        if (ok && n > 0) ok = warp_wait(o_done, (n - 1) & 1);
        if (ok && !idle) {
            tc::tc_fence_after();
            const float g = a.n_split > 1 ? 1.0f : (l == 0.0f ? 0.0f : 1.0f / l);
            const int64_t pr = ((int64_t)z * a.T + tok) * a.q_heads + hq;
            uint16_t* out = a.out + tok * a.out_row_stride + (int64_t)hq * a.out_head_stride;
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
                uint32_t r[16];
                float v[16];
                __syncwarp();
                if (n > 0) {
                    tc::tmem_ld16(tm_o + lanes + 16 * c, r);
                    tc::tmem_ld_wait();
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = (n > 0 && l != 0.0f) ? __uint_as_float(r[i]) * g : 0.0f;
                if (real && a.n_split > 1) {
                    if (l != 0.0f) {
                        float4* dst = reinterpret_cast<float4*>(a.part_o + pr * D + 16 * c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                } else if (real) {
                    uint4* dst = reinterpret_cast<uint4*>(out + 16 * c);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        dst[i] = make_uint4(
                            store_pair<kHalf>(v[8 * i], v[8 * i + 1]), store_pair<kHalf>(v[8 * i + 2], v[8 * i + 3]),
                            store_pair<kHalf>(v[8 * i + 4], v[8 * i + 5]), store_pair<kHalf>(v[8 * i + 6], v[8 * i + 7]));
                }
            }
            if (real) {
                if (a.n_split > 1)
                    a.part_ml[pr] = make_float2(m, l);
                else if (a.lse)
                    a.lse[tok * a.q_heads + hq] = lse_of(m, l);
            }
        }
    } else {
        // ---- converters --------------------------------------------------------------------------------
        const int ct = tid - 128, cw = ct >> 5;
        constexpr int kPieces = D / 16;          // 16-byte pieces of K per thread
        constexpr int kVB = D / 8;               // bytes of V per key and thread: 16 or 8
        const int P = a.page_size, lp = P == 128 ? 7 : 6;
        const int64_t hb = kv_head_bytes(P, D);
        const uint8_t* pool = a.pool + (int64_t)head * hb;
        const int32_t* pt = a.page_table + (int64_t)b * a.pt_stride;
        int64_t* offs = reinterpret_cast<int64_t*>(sm + S::kOff);
        const int vis_sel = kSel ? (int)visible_keys(s.len, s.nq, tok0 - s.t0, a.causal) : 0;
        // K: keys 8 * (cw + 4i) + lane % 8, pieces lane / 8 (+ 4); V: keys 8 * kg .. + 7, dims of dg
        const int kg = (lane & 7) + 8 * (cw & 1), dg = (lane >> 3) + 4 * (cw >> 1);
        uint4 rk[kPieces], rv[8];
        float4 my_scale = make_float4(1.0f, neg_inf(), 0.0f, 0.0f);
        bool bad = false;

        // With a list, thread ct looks up entry ct of a step: the entry two steps ahead, its page one
        // step ahead, its row's place for the loads.
        int32_t ent_n = -1, ent = -1, page = -1;
        int32_t pages[2] = {-1, -1};  // dense: the step's pages (the second for P = 64)
        auto load_entry = [&](int j) -> int32_t {
            const int e = k0 + j * kKeysT + ct;
            return (j < n && e < k1) ? a.sel[tok0 * a.sel_stride + e] : -1;
        };
        auto lookup = [&](int j) {  // pages of step j
            if constexpr (kSel) {
                page = (ent >= 0 && ent < vis_sel) ? pt[ent >> lp] : -1;
            } else {
                const int kt = k0 + j * kKeysT;
                pages[0] = j < n ? pt[kt >> lp] : -1;
                pages[1] = P == 128 ? pages[0] : ((j < n && kt + 64 < k1) ? pt[(kt >> 6) + 1] : -1);
            }
        };
        // where step j's keys are, and the scales (kept in registers until the tile is written)
        auto place = [&](int j) {
            int64_t at = -1;
            int tok = 0;
            if constexpr (kSel) {
                const bool seen = ent >= 0 && ent < vis_sel;
                if (seen && (uint32_t)page >= (uint64_t)a.num_pages) bad = true;
                if (seen && (uint32_t)page < (uint64_t)a.num_pages) {
                    tok = ent & (P - 1);
                    at = (int64_t)page * a.page_stride;
                }
                // the places of step j - 2 have been read: conv_all() came since
                offs[(j & 1) * kKeysT + ct] = at < 0 ? -1 : at + (int64_t)tok * 2 * D;
                conv_sync();
            } else {
                const int key = k0 + j * kKeysT + ct;
                const int32_t pg = pages[P == 64 && ct >= 64];
                if (j < n && key < k1) {
                    if ((uint32_t)pg < (uint64_t)a.num_pages)
                        at = (int64_t)pg * a.page_stride;
                    else
                        bad = true;
                }
                tok = key & (P - 1);
            }
            my_scale = make_float4(1.0f, neg_inf(), 0.0f, 0.0f);
            if (at >= 0 && (kSel || (ct & 15) == 0)) {
                const uint32_t two = *reinterpret_cast<const uint16_t*>(pool + at + 2ll * P * D + 2 * (tok / kKvBlock));
                const float ev = v_exponent(two);
                my_scale = make_float4(k_scale(two), ev, ex2(-ev), 0.0f);
            }
        };
        auto row_of = [&](int j, int key) -> const uint8_t* {  // key's 2*D bytes, or null
            if constexpr (kSel) {
                const int64_t at = offs[(j & 1) * kKeysT + key];
                return at < 0 ? nullptr : pool + at;
            } else {
                const int32_t pg = pages[P == 64 && key >= 64];
                const int at = k0 + j * kKeysT + key;
                if (j >= n || at >= k1 || (uint32_t)pg >= (uint64_t)a.num_pages) return nullptr;
                return pool + (int64_t)pg * a.page_stride + (int64_t)(at & (P - 1)) * 2 * D;
            }
        };
        auto load_k = [&](int j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t* src = row_of(j, 8 * (cw + 4 * i) + (lane & 7));
#pragma unroll
                for (int x = 0; x < D / 64; ++x) {
                    rk[i * (D / 64) + x] = make_uint4(0, 0, 0, 0);
                    if (src) rk[i * (D / 64) + x] = reinterpret_cast<const uint4*>(src)[(lane >> 3) + 4 * x];
                }
            }
        };
        auto load_v = [&](int j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint8_t* src = row_of(j, 8 * kg + i);
                rv[i] = make_uint4(0, 0, 0, 0);
                if (src) {
                    if constexpr (D == 128) {
                        rv[i] = *reinterpret_cast<const uint4*>(src + D + 16 * dg);
                    } else {
                        const uint2 w = *reinterpret_cast<const uint2*>(src + D + 8 * dg);
                        rv[i].x = w.x;
                        rv[i].y = w.y;
                    }
                }
            }
        };
        auto write_k = [&](int j, const float4& sc) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = 8 * (cw + 4 * i) + (lane & 7);
#pragma unroll
                for (int x = 0; x < D / 64; ++x) {
                    const uint4 w = rk[i * (D / 64) + x];
                    uint4 lo, hi;
                    e4m3x4_to_f16x4(w.x, lo.x, lo.y);
                    e4m3x4_to_f16x4(w.y, lo.z, lo.w);
                    e4m3x4_to_f16x4(w.z, hi.x, hi.y);
                    e4m3x4_to_f16x4(w.w, hi.z, hi.w);
                    uint8_t* row = sm + S::kK + x * (kKeysT * 128) + key * 128;
                    const int kc = 2 * (lane >> 3);
                    *reinterpret_cast<uint4*>(row + ((kc ^ (key & 7)) << 4)) = lo;
                    *reinterpret_cast<uint4*>(row + (((kc + 1) ^ (key & 7)) << 4)) = hi;
                }
            }
            if constexpr (kSel)
                scales[(j & 1) * kKeysT + ct] = sc;
            else if ((ct & 15) == 0)
                scales[(j & 1) * kKeysT + ct / 16] = sc;
            tc::fence_proxy_async();
            tc::mbar_arrive(k_full);
        };
        auto write_v = [&]() {
#pragma unroll
            for (int w = 0; w < kVB / 4; ++w) {
                uint32_t u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = w == 0 ? rv[i].x : w == 1 ? rv[i].y : w == 2 ? rv[i].z : rv[i].w;
                uint32_t t[4][4];  // [dim][pair of keys]
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    e4m3x4_to_f16x4(__byte_perm(u[2 * i], u[2 * i + 1], 0x5140), t[0][i], t[1][i]);
                    e4m3x4_to_f16x4(__byte_perm(u[2 * i], u[2 * i + 1], 0x7362), t[2][i], t[3][i]);
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int dim = kVB * dg + 4 * w + y;
                    *reinterpret_cast<uint4*>(sm + S::kV + (kg >> 3) * (D * 128) + dim * 128 +
                                              (((kg & 7) ^ (dim & 7)) << 4)) =
                        make_uint4(t[y][0], t[y][1], t[y][2], t[y][3]);
                }
            }
            tc::fence_proxy_async();
            tc::mbar_arrive(v_full);
        };
        // the MMAs of a step, by one thread
        const bool issuer = warp == 7 && lane == 0;
        const uint32_t base = tc::smem_u32(sm);
        auto issue_s = [&]() {
            tc::tc_fence_after();
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t at = (k / 4) * (128 * 128) + (k % 4) * 32;
                tc::mma_f16(tm_s, tc::smem_desc_sw128(base + S::kQ + at), tc::smem_desc_sw128(base + S::kK + at),
                            tc::idesc_f16(kRowsT, kKeysT), k > 0);
            }
            tc::mma_commit(s_full);
        };
        auto issue_o = [&](bool accumulate) {
            tc::tc_fence_after();
#pragma unroll
            for (int k = 0; k < kKeysT / 16; ++k)
                tc::mma_f16_ta(tm_o, tm_s + 8 * k,
                               tc::smem_desc_sw128(base + S::kV + (k / 4) * (D * 128) + (k % 4) * 32),
                               tc::idesc_f16(kRowsT, D), accumulate || k > 0);
            tc::mma_commit(o_done);
        };

        if (n > 0) {
            if constexpr (kSel) {
                ent = load_entry(0);
                ent_n = load_entry(1);
            }
            lookup(0);
            place(0);
            load_k(0);
            load_v(0);
            float4 sc = my_scale;
            if constexpr (kSel) {
                ent = ent_n;
                ent_n = load_entry(2);
            }
            lookup(1);
            write_k(0, sc);
            if (issuer) {
                ok = tc::mbar_wait(q_full, 0) && tc::mbar_wait(k_full, 0);
                if (ok) issue_s();
            }
            ok = __all_sync(kFull, ok);
            write_v();
            place(1);
            load_k(1);
            load_v(1);
            for (int j = 0; j < n; ++j) {
                // K of step j + 1 goes where step j's product has read; its V where O += P V has
                if (j + 1 < n) {
                    ok = warp_wait(s_full, j & 1) && ok;
                    if constexpr (kSel) ok = conv_all(ok);  // leave together: place() has a barrier
                    if (!ok) break;
                    sc = my_scale;
                    if constexpr (kSel) {
                        ent = ent_n;
                        ent_n = load_entry(j + 3);
                    }
                    lookup(j + 2);
                    write_k(j + 1, sc);
                }
                if (issuer && ok) {
                    ok = tc::mbar_wait(v_full, j & 1) && tc::mbar_wait(p_full, j & 1);
                    if (ok) issue_o(j > 0);
                    // P lies where the next S goes: its product has to be done
                    if (ok && j + 1 < n) {
                        ok = tc::mbar_wait(k_full, (j + 1) & 1) && tc::mbar_wait(o_done, j & 1);
                        if (ok) issue_s();
                    }
                }
                ok = __all_sync(kFull, ok);
                if (j + 1 < n) {
                    ok = warp_wait(o_done, j & 1) && ok;
                    if (!kSel && !ok) break;
                    write_v();
                    place(j + 2);
                    load_k(j + 2);
                    load_v(j + 2);
                }
            }
            if (issuer) {  // what was issued has to finish before the tensor memory is given back
                tc::mma_commit(drain);
                if (!tc::mbar_wait(drain, 0)) ok = false;
            }
            __syncwarp();
        }
        if (bad) report(a.dev_status, IDX_STATUS_BAD_PAGE);
    }
    if (!ok) report(a.dev_status, IDX_STATUS_TIMEOUT);
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 7) tc::tmem_dealloc(tm_s, 256);
}

template <int D, bool kHalf, bool kSel>
cudaError_t launch_tile(const AttnArgs& a, cudaStream_t st) {
    constexpr int smem = SmemT<D>::kBytes;
    auto* kernel = attn_tile_kernel<D, kHalf, kSel>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t units = kSel ? a.T * ((a.group + kRowsT - 1) / kRowsT)
                               : a.B * (((int64_t)a.max_q_len * a.group + kRowsT - 1) / kRowsT);
    return launch_pdl(kernel, dim3((unsigned)units, (unsigned)a.kv_heads, (unsigned)a.n_split), dim3(kThreadsT), smem, st,
                      a);
}

}  // namespace

cudaError_t launch_attn_tile(const AttnArgs& a, cudaStream_t st) {
    if (a.head_dim == 128) {
        if (a.ftype == IDX_FP16) return a.sel ? launch_tile<128, true, true>(a, st) : launch_tile<128, true, false>(a, st);
        return a.sel ? launch_tile<128, false, true>(a, st) : launch_tile<128, false, false>(a, st);
    }
    if (a.ftype == IDX_FP16) return a.sel ? launch_tile<64, true, true>(a, st) : launch_tile<64, true, false>(a, st);
    return a.sel ? launch_tile<64, false, true>(a, st) : launch_tile<64, false, false>(a, st);
}

}  // namespace idx
