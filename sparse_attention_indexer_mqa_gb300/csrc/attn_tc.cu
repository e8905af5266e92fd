// attn_tc.cu -- attention over the 8-bit paged KV cache for many query rows per kv head (prefill, chunks,
// large groups of heads) on the tensor cores with tensor-memory accumulators.
//
// A unit is a tile of 128 query rows of one kv head (token-major: row = token * group + head of the
// group; with a list of keys, the group's heads of one token) against a range of keys, 64 at a time:
// S = Q K^T (M = 128 rows, N = 64 keys), the running softmax of attn.cuh, O += P V (N = D). Tensor memory holds
// two S (the next step's is computed under this step's softmax) and O, 128 + D columns; P overwrites its
// S as fp16 and is the second product's A operand from there. Roles of a CTA's three warpgroups:
//   0  softmax: thread = row, the step's scores in registers. Q to shared memory at the start, O out at the
//      end;
//   1  converters: e4m3 from memory to fp16 operand tiles in shared memory (exact), two stages ahead of the
//      products. The loads go to registers a step before, so any row order costs the same: pages and lists
//      of keys need no gather pass. V is transposed on the way (8 keys x D/16 dims per thread, bytes paired by
//      prmt), which makes both products K-major;
//   2  one warp issues the MMAs.
// fp16 runs at half the 8-bit rate, but 8-bit operands would leave q and the weights 4 bits; two
// 8-bit halves each would cost the same tensor time and more conversion. Two CTAs share an SM
// (tensor memory 2 x 256 columns, shared memory 2 x 101 KB).
#include "attn_tc.cuh"

namespace idx {

namespace {

constexpr int kThreadsT = 384;
// Registers per thread: 80 at launch (two CTAs of 384 threads to an SM); the third warpgroup, of which one
// warp works, gives to the first two: 112 + 88 + 40 = 3 * 80.
constexpr int kRegsSoft = 112, kRegsConv = 88, kRegsIssue = 40;
template <int kRegs>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }

template <int D>
struct SmemT {
    static constexpr int kTile = kKeysT * D * 2;            // bytes of a K or V tile
    static constexpr int kQ = 0;                            // [D/64][128 rows][128 B]
    static constexpr int kK = kQ + kRowsT * D * 2;          // two stages
    static constexpr int kV = kK + 2 * kTile;               // two stages
    static constexpr int kScale = kV + 2 * kTile;           // [4][64] float4: 2^Ek, Ev, 2^-Ev
    static constexpr int kOff = kScale + 4 * kKeysT * 16;   // [2][64] int64: a listed key's row in the pool
    static constexpr int kKey = kOff + 2 * kKeysT * 8;      // [2][64] scale bytes of the listed keys
    static constexpr int kRange = kKey + 2 * kKeysT * 4;    // [2][2] their ranges, a word per warp
    static constexpr int kBar = kRange + 16;
    static constexpr int kBytes = kBar + 128 + 1024;        // 1024: alignment of the operand tiles
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
template <int D, bool kHalf, bool kSel>
__global__ void __launch_bounds__(kThreadsT, 2) attn_tile_kernel(const AttnArgs a) {
    using S = SmemT<D>;
    extern __shared__ uint8_t sm_raw[];
    __shared__ uint32_t tmem_slot;
    uint8_t* sm = sm_raw + ((1024u - (tc::smem_u32(sm_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::kBar);
    // one of each per parity of the step (and so per stage): who waits for a step may find that the
    // next one's has come, but not the one's after it
    uint64_t *k_full = bars, *v_full = bars + 2, *s_full = bars + 4, *p_full = bars + 6, *o_done = bars + 8,
             *q_full = bars + 10, *drain = bars + 11;
    float4* scales = reinterpret_cast<float4*>(sm + S::kScale);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

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
    if (tid == 0) {
        tc::mbar_init(q_full, kRowsT);
        tc::mbar_init(drain, 1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(k_full + i, 128);
            tc::mbar_init(v_full + i, 128);
            tc::mbar_init(s_full + i, 1);
            tc::mbar_init(p_full + i, (rows + 31) / 32);  // a warp without rows takes no part
            tc::mbar_init(o_done + i, 1);
        }
        tc::fence_mbar_init();
    }
    __syncwarp();
    if (warp == 8) {
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
        regs_up<kRegsSoft>();
        const bool real = tid < rows;
        const int row = row0 + min(tid, rows - 1);
        const int64_t tok = kSel ? tok0 : tok0 + row / G;
        const int hq = head * G + (kSel ? row : row % G);
        const int vis = (int)visible_keys(s.len, s.nq, tok - s.t0, a.causal);
        const float rc = write_q_row<D, kHalf>(sm + S::kQ, a.q + tok * a.q_row_stride + (int64_t)hq * a.q_head_stride,
                                               real, tid, a.scale);
        tc::mbar_arrive(q_full);
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const bool idle = 32 * warp >= rows;  // no row of this warp exists
        float m = neg_inf(), l = 0.0f;
        // A row whose largest u passes m by more than kLazy: m raised, O (complete up to the step before) and
        // l scaled.
        auto raise_to = [&](int j, float mx) {
            float f = 1.0f;
            const bool raise = mx > m + kLazy;
            if (raise) {
                f = ex2(m - mx);
                m = mx;
                l *= f;
            }
            if (j > 0 && __any_sync(kFull, raise)) {
                ok = warp_wait<kNsSoft>(o_done + ((j - 1) & 1), ((j - 1) >> 1) & 1) && ok;
                tc::tc_fence_after();
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
        };
        // One step of the running softmax, S to P, with a scale pair per 16 keys; the row's scores stay in
        // registers. kCut: the rows' visibility tested key by key (tiles that some row of the warp does not
        // see whole).
        auto step = [&](int j, auto cut_tag) {
            constexpr bool kCut = decltype(cut_tag)::value;
            const uint32_t tm = tm_s + kKeysT * (j & 1) + lanes;
            const float4* sc = scales + (j & 3) * kKeysT;
            [[maybe_unused]] const int left = vis - (k0 + j * kKeysT);  // keys of this step that the row sees
            uint32_t r[2][32];
            __syncwarp();
            tc::tmem_ld32(tm, r[0]);
            tc::tmem_ld32(tm + 32, r[1]);
            tc::tmem_ld_wait();
            float mx = neg_inf();
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const uint32_t* x = &r[h >> 1][16 * (h & 1)];
                const float4 k = sc[h];
                float bm = neg_inf();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    bm = fmaxf(bm, !kCut || 16 * h + i < left ? __uint_as_float(x[i]) : neg_inf());
                // nothing visible: bm is -inf whatever the factor
                const float u = fmaf(bm, rc * k.x, k.y);
                mx = fmaxf(mx, kCut && bm == neg_inf() ? bm : u);
            }
            raise_to(j, mx);
            const float top = m == neg_inf() ? 0.0f : kShift - m;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint32_t p2[16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t* x = &r[g][16 * h];
                    const float4 k = sc[2 * g + h];
                    const float cc = rc * k.x, sub = k.y + top;
                    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        float2 u = fma2(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), make_float2(cc, cc),
                                        make_float2(sub, sub));
                        if constexpr (kCut) {
                            u.x = 32 * g + 16 * h + i < left ? u.x : neg_inf();
                            u.y = 32 * g + 16 * h + i + 1 < left ? u.y : neg_inf();
                        }
                        const float2 p = make_float2(ex2(u.x), ex2(u.y));
                        sum = add2(sum, p);
                        p2[8 * h + i / 2] = half2_bits(p.x, p.y);
                    }
                    l = fmaf(sum.x + sum.y, k.z, l);
                }
                tc::tmem_st16(tm + 16 * g, p2);
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
        };
        // The same with a scale pair per key (lists), Ev = -inf where a key does not count; 16 keys at a time.
        auto step_keyed = [&](int j) {
            const uint32_t tm = tm_s + kKeysT * (j & 1) + lanes;
            const float4* sc = scales + (j & 3) * kKeysT;
            float mx = neg_inf();
#pragma unroll 1
            for (int c = 0; c < kKeysT / 16; ++c) {
                uint32_t r[16];
                __syncwarp();
                tc::tmem_ld16(tm + 16 * c, r);
                tc::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float4 k = sc[16 * c + i];
                    mx = fmaxf(mx, fmaf(__uint_as_float(r[i]), rc * k.x, k.y));
                }
            }
            raise_to(j, mx);
            const float top = m == neg_inf() ? 0.0f : kShift - m;
#pragma unroll 1
            for (int c = 0; c < kKeysT / 16; ++c) {
                uint32_t r[16], p2[8];
                __syncwarp();
                tc::tmem_ld16(tm + 16 * c, r);
                tc::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float4 ka = sc[16 * c + i], kb = sc[16 * c + i + 1];
                    const float pa = ex2(fmaf(__uint_as_float(r[i]), rc * ka.x, ka.y + top));
                    const float pb = ex2(fmaf(__uint_as_float(r[i + 1]), rc * kb.x, kb.y + top));
                    l = fmaf(pa, ka.z, l);
                    l = fmaf(pb, kb.z, l);
                    p2[i / 2] = half2_bits(pa, pb);
                }
                tc::tmem_st8(tm + 8 * c, p2);  // columns that have been read
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
        };
        for (int j = 0; j < n && !idle; ++j) {
            ok = warp_wait<kNsSoft>(s_full + (j & 1), (j >> 1) & 1);
            if (!ok) break;
            tc::tc_fence_after();
            if constexpr (kSel) {
                if (scales[(j & 3) * kKeysT].w != 0.0f)
                    step_keyed(j);
                else
                    step(j, std::false_type{});
            } else {
                if (__any_sync(kFull, k0 + (j + 1) * kKeysT > vis))
                    step(j, std::true_type{});
                else
                    step(j, std::false_type{});
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(p_full + (j & 1));
            if (!ok) break;
        }
        // ---- the row's result -------------------------------------------------------------------------
        if (ok && n > 0 && !idle) ok = warp_wait<kNsSoft>(o_done + ((n - 1) & 1), ((n - 1) >> 1) & 1);
        if (ok && !idle) {
            tc::tc_fence_after();
            store_rows<D, kHalf>(a, tm_o + lanes, n > 0, real, tok, hq, z, m, l);
        }
    } else if (warp < 8) {
        // ---- converters --------------------------------------------------------------------------------
        regs_up<kRegsConv>();
        const int ct = tid - 128, cw = ct >> 5;
        using C = ConvShare<D>;
        const C my(ct);
        constexpr int kPieces = C::kPieces;
        const int P = a.page_size, lp = P == 128 ? 7 : 6;
        const int64_t hb = kv_head_bytes(P, D);
        const uint8_t* pool = a.pool + (int64_t)head * hb;
        const int32_t* pt = a.page_table + (int64_t)b * a.pt_stride;
        int64_t* offs = reinterpret_cast<int64_t*>(sm + S::kOff);
        const int vis_sel = kSel ? (int)visible_keys(s.len, s.nq, tok0 - s.t0, a.causal) : 0;
        uint4 rk[kPieces];
        uint2 rv[8];
        uint32_t my_scale = 0;  // the key's or block's two scale bytes, bit 16 set; 0: not to be used
        bool bad = false;

        // Lookups run ahead: a step's page is loaded one step before its rows, and with a list (thread ct
        // looks after entry ct of a step) its entry two steps before.
        int32_t ent = -1, ent_n = -1, page = -1;
        const uint8_t* rows_at = nullptr;  // key 0 of the step
        int keys = 0;                      // of the step
        auto load_entry = [&](int j) -> int32_t {
            const int e = k0 + j * kKeysT + ct;
            return ct < kKeysT && e < k1 ? a.sel[tok0 * a.sel_stride + e] : -1;
        };
        auto lookup = [&](int j) {
            if constexpr (kSel) {
                page = (ent >= 0 && ent < vis_sel) ? pt[ent >> lp] : -1;
            } else {
                const int kt = k0 + j * kKeysT;
                page = kt < k1 ? pt[kt >> lp] : -1;
            }
        };
        auto place = [&](int j) {
            const bool in = (uint32_t)page < (uint64_t)a.num_pages;
            my_scale = 0;
            if constexpr (kSel) {
                const bool seen = ent >= 0 && ent < vis_sel;
                int64_t at = -1;
                bad |= seen && !in;
                if (seen && in) {
                    const int tok = ent & (P - 1);
                    at = (int64_t)page * a.page_stride;
                    my_scale = *reinterpret_cast<const uint16_t*>(pool + at + 2ll * P * D + 2 * (tok / kKvBlock)) | 65536u;
                    at += (int64_t)tok * 2 * D;
                }
                // the places of step j - 2 have been read: conv_all() came since
                if (ct < kKeysT) offs[(j & 1) * kKeysT + ct] = at;
                conv_sync();
            } else {
                const int kt = k0 + j * kKeysT, tok = kt & (P - 1);
                keys = k1 - kt;
                bad |= !in;
                const uint8_t* at = pool + (int64_t)page * a.page_stride;
                if (in && (ct & 15) == 0 && ct < kKeysT && ct < keys)  // this thread's block of 16 keys
                    my_scale = *reinterpret_cast<const uint16_t*>(at + 2ll * P * D + 2 * ((tok + ct) / kKvBlock)) | 65536u;
                rows_at = in ? at + tok * 2 * D : nullptr;
            }
        };
        auto load_k = [&](int j) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int key = my.k_key + C::kKeyStep * i;
                const uint8_t* src = rows_at + key * 2 * D;
                bool in = rows_at != nullptr && key < keys;
                if constexpr (kSel) {
                    const int64_t at = offs[(j & 1) * kKeysT + key];
                    src = pool + at;
                    in = at >= 0;
                }
                uint4 w = make_uint4(0, 0, 0, 0);
                if (in) w = reinterpret_cast<const uint4*>(src)[my.kp];
                rk[i] = w;
            }
        };
        auto load_v = [&](int j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int key = 8 * my.kg + i;
                const uint8_t* src = rows_at + key * 2 * D;
                bool in = rows_at != nullptr && key < keys;
                if constexpr (kSel) {
                    const int64_t at = offs[(j & 1) * kKeysT + key];
                    src = pool + at;
                    in = at >= 0;
                }
                uint2 w = make_uint2(0, 0);
                if constexpr (D == 128) {
                    if (in) w = *reinterpret_cast<const uint2*>(src + D + 8 * my.dg);
                } else {
                    if (in) w.x = *reinterpret_cast<const uint32_t*>(src + D + 4 * my.dg);
                }
                rv[i] = w;
            }
        };
        // A list's keys have scales of their own. Where a step's lie within 2^15 of one another and every key
        // counts, they are folded into the fp16 operands (exact: a code is at least 2^-9, fp16
        // reaches 2^-24) and the softmax sees one scale pair; otherwise it takes a pair per key.
        uint32_t* key_scales = reinterpret_cast<uint32_t*>(sm + S::kKey);
        uint32_t* ranges = reinterpret_cast<uint32_t*>(sm + S::kRange);
        int k_top = 0, v_top = 0;  // largest scale bytes of the step
        bool fold = false;
        auto publish = [&](int j) {  // before the barrier
            const uint32_t ek = scale_byte(my_scale), ev = scale_byte(my_scale >> 8);
            const bool in = my_scale != 0;
            const uint32_t k_hi = __reduce_max_sync(kFull, in ? ek : 255u), k_lo = __reduce_min_sync(kFull, in ? ek : 0u);
            const uint32_t v_hi = __reduce_max_sync(kFull, in ? ev : 255u), v_lo = __reduce_min_sync(kFull, in ? ev : 0u);
            if (ct < kKeysT) key_scales[(j & 1) * kKeysT + ct] = my_scale;
            if (lane == 0 && cw < 2) ranges[(j & 1) * 2 + cw] = k_hi | k_lo << 8 | v_hi << 16 | v_lo << 24;
        };
        auto collect = [&](int j) {  // behind it
            const uint2 r = *reinterpret_cast<const uint2*>(ranges + (j & 1) * 2);
            const uint32_t hi = __vmaxu4(r.x, r.y), lo = __vminu4(r.x, r.y);
            k_top = hi & 255;
            v_top = hi >> 16 & 255;
            // a key that does not count makes the range too wide
            fold = k_top - (int)(lo >> 8 & 255) <= 15 && v_top - (int)(lo >> 24) <= 15;
        };
        auto down = [&](int by) -> uint32_t {  // 2^-by as fp16 bits, by in 0 .. 15
            return by < 15 ? (uint32_t)(15 - by) << 10 : 0x0200u;
        };
        auto write_k = [&](int j) {
            const float ev = v_exponent(my_scale);
            const float4 sc = my_scale ? make_float4(k_scale(my_scale), ev, ex2(-ev), 1.0f)
                                       : make_float4(1.0f, neg_inf(), 0.0f, 1.0f);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int key = my.k_key + C::kKeyStep * i;
                uint32_t f = 0;
                if constexpr (kSel) {
                    if (fold) f = down(k_top - (int)scale_byte(key_scales[(j & 1) * kKeysT + key])) * 65537u;
                }
                write_k_piece<D>(sm + S::kK + (j & 1) * S::kTile, rk[i], key, my.kp, f);
            }
            // four buffers of scales: a softmax may still read those of the stage's last step
            float4* to = scales + (j & 3) * kKeysT;
            if constexpr (kSel) {
                if (!fold) {
                    if (ct < kKeysT) to[ct] = sc;
                } else if (ct < 4) {
                    to[ct] = make_float4(__uint_as_float((uint32_t)k_top << 23), (float)(v_top - 127),
                                         ex2((float)(127 - v_top)), 0.0f);
                }
            } else if ((ct & 15) == 0 && ct < kKeysT) {
                to[ct / 16] = sc;
            }
            tc::mbar_arrive(k_full + (j & 1));
        };
        auto write_v = [&](int j) {
            uint32_t f[4] = {0, 0, 0, 0};  // factors of pairs of keys
            if constexpr (kSel) {
                if (fold) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint2 two = *reinterpret_cast<const uint2*>(key_scales + (j & 1) * kKeysT + 8 * my.kg + 2 * i);
                        f[i] = down(v_top - (int)scale_byte(two.x >> 8)) | down(v_top - (int)scale_byte(two.y >> 8)) << 16;
                    }
                }
            }
            write_v_block<D>(sm + S::kV + (j & 1) * S::kTile, rv, my.kg, my.dg, kSel && fold, f);
            tc::mbar_arrive(v_full + (j & 1));
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
            if constexpr (kSel) {
                ent = ent_n;
                ent_n = load_entry(2);
            }
            lookup(1);
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
                // a stage's K is free when step j - 2's product has read it, its V when O += P V has
                if (j >= 2) ok = warp_wait<kNsConv>(s_full + (j & 1), ((j - 2) >> 1) & 1) && ok;
                if constexpr (kSel) {
                    publish(j);
                    ok = conv_all(ok);  // leave together: place() has a barrier
                    collect(j);
                }
                if (!ok) break;
                write_k(j);
                if (j + 1 < n) {
                    place(j + 1);
                    load_k(j + 1);
                }
                if (j >= 2) ok = warp_wait<kNsConv>(o_done + (j & 1), ((j - 2) >> 1) & 1) && ok;
                write_v(j);
                if (j + 1 < n) {
                    load_v(j + 1);
                    if constexpr (kSel) {
                        ent = ent_n;
                        ent_n = load_entry(j + 3);
                    }
                    lookup(j + 2);
                }
            }
        }
        if (bad) report(a.dev_status, IDX_STATUS_BAD_PAGE);
    } else {
        // ---- MMA: S of step j, then O += P V of step j - 1 ----------------------------------------------------
        regs_down<kRegsIssue>();
        if (warp == 8 && n > 0) {
            const uint32_t base = tc::smem_u32(sm);
            ok = warp_wait<kNsIssue>(q_full, 0);
            for (int j = 0; j <= n && ok; ++j) {
                const int st = j & 1;
                if (j < n) {
                    // P of step j - 2 lies where this S goes: its product has to be done
                    ok = warp_wait<kNsIssue>(k_full + st, (j >> 1) & 1) &&
                         (j < 2 || warp_wait<kNsIssue>(o_done + st, ((j - 2) >> 1) & 1));
                    if (!ok) break;
                    // The tiles were written with ordinary stores: the proxy fence between those and the MMAs' reads is
                    // here, behind the barrier, because in the converters it would wait for the loads they have in
                    // flight.
                    tc::fence_proxy_async();
                    issue_scores<D>(tm_s + kKeysT * st, base + S::kQ, base + S::kK + st * S::kTile, s_full + st);
                }
                if (j > 0) {
                    const int pv = st ^ 1;
                    ok = warp_wait<kNsIssue>(v_full + pv, ((j - 1) >> 1) & 1) &&
                         warp_wait<kNsIssue>(p_full + pv, ((j - 1) >> 1) & 1);
                    if (!ok) break;
                    tc::fence_proxy_async();
                    issue_outputs<D>(tm_o, tm_s + kKeysT * pv, base + S::kV + pv * S::kTile, j > 1, o_done + pv);
                }
            }
            // what was issued has to finish before the tensor memory is given back
            if (tc::elect_one()) tc::mma_commit(drain);
            __syncwarp();
            ok = warp_wait<kNsIssue>(drain, 0) && ok;
        }
    }
    if (!ok) report(a.dev_status, IDX_STATUS_TIMEOUT);
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 8) tc::tmem_dealloc(tm_s, 256);
}

template <int D, bool kHalf, bool kSel>
cudaError_t launch_tile(const AttnArgs& a, cudaStream_t st) {
    constexpr int smem = SmemT<D>::kBytes;
    auto* kernel = attn_tile_kernel<D, kHalf, kSel>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(allowed, kernel, smem);
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
