// attn_tc.cu -- attention over the 8-bit paged KV cache for many query rows per kv head (prefill, chunks,
// large groups of heads, trees of drafted tokens) on the tensor cores with tensor-memory accumulators.
//
// A unit is a tile of 128 query rows of one kv head (token-major: row = token * group + head of the
// group; with a list of keys, the group's heads of one token) against a range of keys, 128 at a
// time: S = Q K^T (M = 128 rows, N = 128 keys), the running softmax of attn.cuh, O += P V (N = D). S and
// O live in tensor memory (128 + D columns), P overwrites S as fp16 and is the second product's A
// operand from there. Roles of a CTA's two warpgroups:
//   0  softmax: thread = row. Q to shared memory at the start, S -> P per tile, O out at the end; warp
//      0 issues the MMAs, which it would wait for anyway (in a converter warp each step waited for that
//      warp's other work, 674 us for a causal prompt of 8192 tokens, 32 heads over 8, against 630 then; in a
//      warp of its own every thread had a quarter fewer registers and spilled, 898 us);
//   1  converters: e4m3 from memory to fp16 operand tiles in shared memory (exact). The loads of a
//      tile go out one tile ahead into registers, so any row order costs the same: pages and
//      lists of keys need no gather pass. V is transposed on the way (8 keys x 16 dims per
//      thread, bytes paired by prmt), which makes both products K-major.
// fp16 runs at half the 8-bit rate, but 8-bit operands would leave q and the weights 4 bits; two
// 8-bit halves each would cost the same tensor time and more conversion. Two CTAs share an SM
// (tensor memory 2 x 256 columns, shared memory 2 x 107 KB): one's products run under the other's
// softmax.
//
// What bounds it. That prompt takes 588 us, 935 TFLOP/s of its visible pairs (47 % of a large bf16 product's measured
// rate). Eight MMAs of 128 x 128 x 16 take 736 cycles (both operands in shared memory) or 679
// (P in tensor memory) with nothing else on the SM, so a step needs 1415 cycles of the tensor pipe;
// a CTA's step takes 4400: S 740, softmax 1950, O += P V 700, and 200 to 500 from each to
// the next. Measured and no faster: 64-key steps with two S (S of the next step under this step's softmax;
// an N = 64 MMA takes as long as an N = 128 one: 600 us, and 548 with lists, which were at 443 then),
// with K's and V's converters apart (645, 518); two tiles to a CTA that share converted K and V (698, and
// 685 with the tiles' MMAs in turn); the softmax in one pass over S with P kept in registers
// (665). With lists (4096 queries x 1024 keys, 64 heads over 1: 386 us) half of a tile's rows are
// empty and a unit is only eight steps long; the order of the keys hardly matters (447 in order, 453 at random, when the
// converters still looked the keys up).
//
// Trees. 64 requests of 16 nodes on 8176 keys, 64 heads over 8, are 512 units of 128 rows and 65 steps: 338 us, where the cache
// (1.1 GB) takes 164 at the copy rate and the products 139. Each key is read by one unit, from memory: 391 us until it was sent for
// into L2 (send_for), 346 until q and the results moved in whole lines. 304 CTAs fit, so the units take 1.7 rounds and two are
// paid for; a step is 4800 cycles (S 850, softmax 2100, O += P V 900, waits 950) and 5500 with two CTAs on the SM, whose
// shared-memory port is then about three quarters busy (operands written and read, tensor pipe 35 %, ALU 38 %: profiles). Lists of
// 1024 keys and 8 nodes for 64 requests: 80 us, 23 at the copy rate; nine steps a unit and two rounds, a converter's step of
// 5000 cycles, half of it folding scales into operands.
#include "attn_tc.cuh"

namespace idx {

namespace {

constexpr int kThreadsT = 256;
constexpr int kFar = 2;  // see send_for

template <int D>
struct SmemT {
    static constexpr int kQ = 0;                            // [D/64][128 rows][128 B]
    static constexpr int kK = kQ + kRowsT * D * 2;          // [D/64][128 keys][128 B]
    static constexpr int kV = kK + kKeysT * D * 2;          // [2][D dims][128 B]
    static constexpr int kScale = kV + kKeysT * D * 2;      // [2][128] float4: 2^Ek, Ev, 2^-Ev
    static constexpr int kOff = kScale + 2 * kKeysT * 16;   // [2][128] int64: a listed key's row in the pool
    static constexpr int kKey = kOff + 2 * kKeysT * 8;      // [2][128] scale bytes of the listed keys
    static constexpr int kRange = kKey + 2 * kKeysT * 4;    // [2][4] their ranges, a word per warp
    static constexpr int kBar = kRange + 32;
    static constexpr int kBytes = kBar + 80 + 1024;         // 1024: alignment of the operand tiles
    static_assert(kK + kRowsT * kOutRow<D> <= kBar, "results are staged from K's tile on");
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
template <int D, bool kHalf, bool kSel, bool kTree>
__global__ void __launch_bounds__(kThreadsT, 2) attn_tile_kernel(const AttnArgs a) {
    using S = SmemT<D>;
    extern __shared__ uint8_t sm_raw[];
    __shared__ uint32_t tmem_slot;
    // kTree: a bit per node whose V held a NaN code that was taken out, and a word for the keys in front of the tree
    __shared__ uint32_t nan_nodes[kTree && !kSel ? kTreeMaxNodes / 32 + 1 : 1];
    uint8_t* sm = sm_raw + ((1024u - (tc::smem_u32(sm_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::kBar);
    uint64_t *q_full = bars, *k_full = bars + 1, *v_full = bars + 2, *s_full = bars + 3, *p_full = bars + 4,
             *o_done = bars + 5, *drain = bars + 6;
    // [2], steps in turn: a helper may be done with steps 0 and 1 before the other has done step 0
    [[maybe_unused]] uint64_t* look_full = bars + 8;
    int* nan_key = reinterpret_cast<int*>(bars + 7);  // lowest key whose V held a NaN code that was taken out
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
        b = warp_seq_of_query(a, t);
        if (b >= 0) s = seq_rows(a, b);
        row0 = (int)(blockIdx.x % tiles) * kRowsT;
        tok0 = t;
        rows = b < 0 ? 0 : min(kRowsT, G - row0);
        kv_end = a.n_sel + (kTree && b >= 0 ? max(s.nq, 0) : 0);
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
    if (rows <= 0) return;
    if (tid == 0) {
        tc::mbar_init(q_full, kRowsT);
        tc::mbar_init(k_full, 128);
        tc::mbar_init(v_full, 128);
        tc::mbar_init(s_full, 1);
        tc::mbar_init(p_full, (rows + 31) / 32);  // a warp without rows takes no part
        tc::mbar_init(o_done, 1);
        tc::mbar_init(drain, 1);
        tc::mbar_init(look_full, 2);
        tc::mbar_init(look_full + 1, 2);
        *nan_key = INT32_MAX;
        tc::fence_mbar_init();
    }
    if constexpr (kTree && !kSel) {
        if (tid <= kTreeMaxNodes / 32) nan_nodes[tid] = 0;
    }
    __syncwarp();
    if (warp == 0) {
        tc::tmem_alloc(&tmem_slot, 256);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (a.n_split > 1) pdl_launch_dependents();  // the join
    const uint32_t tm_s = tmem_slot, tm_o = tm_s + 128;
    const int k0 = z * a.chunk, k1 = min(kv_end, k0 + a.chunk);
    const int n = k1 > k0 ? (k1 - k0 + kKeysT - 1) / kKeysT : 0;
    bool ok = true;
    [[maybe_unused]] const int front = s.len - s.nq;  // keys in front of the tree
    // A list's lookups: with up to 64 rows by the softmax warps that have none.
    const bool helped = kSel && rows <= 64;
    int64_t* offs = reinterpret_cast<int64_t*>(sm + S::kOff);
    uint32_t* key_scales = reinterpret_cast<uint32_t*>(sm + S::kKey);
    uint32_t* ranges = reinterpret_cast<uint32_t*>(sm + S::kRange);
    const int P = a.page_size, lp = P == 128 ? 7 : 6;
    const uint8_t* pool = a.pool + (int64_t)head * kv_head_bytes(P, D);
    const int32_t* pt = a.page_table + (int64_t)b * a.pt_stride;
    const int vis_sel = kSel ? (int)visible_keys(s.len, s.nq, tok0 - s.t0, a.causal) : 0;
    // Entry i of step j, and whether what it holds counts.
    auto load_entry = [&](int j, int i) -> int32_t {
        const int e = k0 + j * kKeysT + i;
        if constexpr (kTree) {  // the nodes that the row sees come behind its list
            const int node = e - a.n_sel;
            if (node >= 0)
                return e < k1 && tree_window(a.tree + tok0 * a.tree_stride, a.tree_words, s.nq, node) & 1 ? front + node : -1;
        }
        return e < k1 ? a.sel[tok0 * a.sel_stride + e] : -1;
    };
    auto counts = [&](int j, int i, int32_t ent) -> bool {
        const int end = kTree && k0 + j * kKeysT + i < a.n_sel ? front : vis_sel;
        return ent >= 0 && ent < end;
    };
    // The ranges of the scale bytes that a warp's lanes give (two each), a byte each from the lowest on: largest K, smallest K,
    // largest V, smallest V. The caller puts the word among the step's four.
    auto ranges_of = [&](uint32_t lo_scale, uint32_t hi_scale) -> uint32_t {
        uint32_t k_hi = 0, k_lo = 255, v_hi = 0, v_lo = 255;
        // a key that does not count makes the range too wide
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t two = i ? hi_scale : lo_scale, ek = scale_byte(two), ev = scale_byte(two >> 8);
            k_hi = max(k_hi, two ? ek : 255u);
            k_lo = min(k_lo, two ? ek : 0u);
            v_hi = max(v_hi, two ? ev : 255u);
            v_lo = min(v_lo, two ? ev : 0u);
        }
        return __reduce_max_sync(kFull, k_hi) | __reduce_min_sync(kFull, k_lo) << 8 | __reduce_max_sync(kFull, v_hi) << 16 |
               __reduce_min_sync(kFull, v_lo) << 24;
    };

    if (warp < 4) {
        // ---- softmax: this thread's row --------------------------------------------------------------
        const bool real = tid < rows;
        const int row = row0 + min(tid, rows - 1);
        const int64_t tok = kSel ? tok0 : tok0 + row / G;
        const int hq = head * G + (kSel ? row : row % G);
        // keys that the row sees, of a tree: those in front of it
        const int vis = kTree && !kSel ? front : (int)visible_keys(s.len, s.nq, tok - s.t0, a.causal);
        [[maybe_unused]] const uint64_t* mask = kTree ? a.tree + tok * a.tree_stride : nullptr;
        // < 0: an infinity or a NaN in q; the row is scored as zeros, and is NaN at the end if any key counted
        const float rc = write_q_rows<D, kHalf>(sm + S::kQ, a.q + tok * a.q_row_stride + (int64_t)hq * a.q_head_stride,
                                                real, 32 * warp, a.scale);
        tc::fence_proxy_async();
        tc::mbar_arrive(q_full);
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const bool idle = 32 * warp >= rows;  // no row of this warp exists
        float m = neg_inf(), l = 0.0f;
        // A row whose largest u passes m by more than kLazy: m raised, O and l scaled.
        auto raise_to = [&](int j, float mx) {
            float f = 1.0f;
            const bool raise = mx > m + kLazy;
            if (raise) {
                f = ex2(m - mx);
                m = mx;
                l *= f;
            }
            if (j > 0 && __any_sync(kFull, raise)) {
                // the scores were issued behind the completed O += P V of the step before
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t r[2][16];
                    __syncwarp();
                    tc::tmem_ld16(tm_o + lanes + 32 * c, r[0]);
                    tc::tmem_ld16(tm_o + lanes + 32 * c + 16, r[1]);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        r[0][i] = __float_as_uint(__uint_as_float(r[0][i]) * f);
                        r[1][i] = __float_as_uint(__uint_as_float(r[1][i]) * f);
                    }
                    tc::tmem_st16(tm_o + lanes + 32 * c, r[0]);
                    tc::tmem_st16(tm_o + lanes + 32 * c + 16, r[1]);
                }
            }
        };
        // One step of the running softmax, S to P, with a scale pair per 16 keys. kCut: the rows' visibility
        // tested key by key (tiles that some row of the warp does not see whole).
        auto step = [&](int j, auto cut_tag) {
            constexpr bool kCut = decltype(cut_tag)::value;
            const float4* sc = scales + (j & 1) * kKeysT;
            [[maybe_unused]] const int left = vis - (k0 + j * kKeysT);  // keys of this step that the row sees
            // of a tree: which ones of 64
            [[maybe_unused]] auto window = [&](int from) { return tree_window(mask, a.tree_words, s.nq, from - left); };
            float mx = neg_inf();
#pragma unroll 1
            for (int c = 0; c < 4; c += 2) {
                uint32_t r[2][32];
                __syncwarp();
                tc::tmem_ld32(tm_s + lanes + 32 * c, r[0]);
                tc::tmem_ld32(tm_s + lanes + 32 * c + 32, r[1]);
                [[maybe_unused]] uint64_t shown = 0;
                if constexpr (kTree && kCut) shown = window(32 * c);
                tc::tmem_ld_wait();
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const uint32_t* x = &r[h >> 1][16 * (h & 1)];
                    const int at = 32 * c + 16 * h;
                    const float4 k = sc[at / 16];
                    float bm = neg_inf();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const bool in = !kCut || (kTree ? shown >> (16 * h + i) & 1 : at + i < left);
                        bm = fmaxf(bm, in ? __uint_as_float(x[i]) : neg_inf());
                    }
                    // nothing visible: bm is -inf whatever the factor
                    const float u = fmaf(bm, rc * k.x, k.y);
                    mx = fmaxf(mx, kCut && bm == neg_inf() ? bm : u);
                }
            }
            raise_to(j, mx);
            const float top = m == neg_inf() ? 0.0f : kShift - m;
#pragma unroll 1
            for (int c = 0; c < 4; c += 2) {
                uint32_t r[2][32];
                __syncwarp();
                tc::tmem_ld32(tm_s + lanes + 32 * c, r[0]);
                tc::tmem_ld32(tm_s + lanes + 32 * c + 32, r[1]);
                [[maybe_unused]] uint64_t shown = 0;
                if constexpr (kTree && kCut) shown = window(32 * c);
                tc::tmem_ld_wait();
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    uint32_t p2[16];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t* x = &r[g][16 * h];
                        const int at = 32 * (c + g) + 16 * h;
                        const float4 k = sc[at / 16];
                        const float cc = rc * k.x, sub = k.y + top;
                        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            float2 u = fma2(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])),
                                            make_float2(cc, cc), make_float2(sub, sub));
                            if constexpr (kCut) {
                                const int bit = 32 * g + 16 * h + i;
                                u.x = (kTree ? shown >> bit & 1 : at + i < left) ? u.x : neg_inf();
                                u.y = (kTree ? shown >> (bit + 1) & 1 : at + i + 1 < left) ? u.y : neg_inf();
                            }
                            const float2 p = make_float2(ex2(u.x), ex2(u.y));
                            sum = add2(sum, p);
                            p2[8 * h + i / 2] = half2_bits(p.x, p.y);
                        }
                        l = fmaf(sum.x + sum.y, k.z, l);
                    }
                    // columns 16(c+g) .. +15 held scores that have been read
                    tc::tmem_st16(tm_s + lanes + 16 * (c + g), p2);
                }
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
        };
        // The same with a scale pair per key (lists), Ev = -inf where a key does not count. 16 keys at a
        // time: more registers would spill, and reloads that miss L1 hold up the thread that issues
        // the MMAs.
        auto step_keyed = [&](int j) {
            const float4* sc = scales + (j & 1) * kKeysT;
            float mx = neg_inf();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
                uint32_t r[16];
                __syncwarp();
                tc::tmem_ld16(tm_s + lanes + 16 * c, r);
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
            for (int c = 0; c < 8; ++c) {
                uint32_t r[16], p2[8];
                __syncwarp();
                tc::tmem_ld16(tm_s + lanes + 16 * c, r);
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
                tc::tmem_st8(tm_s + lanes + 8 * c, p2);  // columns that have been read
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
        };
        // A list's lookups by the warps of rows 64 .. 127 where there are none: for each step the places of its keys' rows and
        // the scale bytes, two entries a thread. In the converters they were half of a round's chain of instructions (a step
        // of 7500 cycles; the products and the softmax take 4800). Step j + 2's places lie where step j's were.
        if constexpr (kSel) {
            if (helped && warp >= 2) {
                const int ht = tid - 64;
                int32_t ent[2], pg[2];
                int64_t at[2], at_n[2];
                uint32_t two[2], two_n[2];
                bool bad = false;
                auto look = [&](int j) {  // pages of step j, whose entries are there
#pragma unroll
                    for (int i = 0; i < 2; ++i) pg[i] = j < n && counts(j, ht + 64 * i, ent[i]) ? pt[ent[i] >> lp] : -1;
                };
                auto place = [&](int j) {  // places and scales of step j, whose pages are there
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const bool seen = j < n && counts(j, ht + 64 * i, ent[i]), in = (uint32_t)pg[i] < (uint64_t)a.num_pages;
                        bad |= seen && !in;
                        at_n[i] = -1;
                        two_n[i] = 0;
                        if (seen && in) {
                            const int tok = ent[i] & (P - 1);
                            at_n[i] = (int64_t)pg[i] * a.page_stride;
                            two_n[i] = *reinterpret_cast<const uint16_t*>(pool + at_n[i] + 2ll * P * D + 2 * (tok / kKvBlock)) | 65536u;
                            at_n[i] += (int64_t)tok * 2 * D;
                            if constexpr (kTree) {  // read by few units, as a dense tree's keys are: see send_for
#pragma unroll
                                for (int line = 0; line < 2 * D; line += 128)
                                    asm volatile("prefetch.global.L2 [%0];" ::"l"(pool + at_n[i] + line));
                            }
                        }
                    }
                };
                auto entries = [&](int j) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) ent[i] = j < n ? load_entry(j, ht + 64 * i) : -1;
                };
                entries(0);
                look(0);
                place(0);
                entries(1);
                look(1);
#pragma unroll 1
                for (int j = 0; j < n; ++j) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        at[i] = at_n[i];
                        two[i] = two_n[i];
                    }
                    if (j >= 2) ok = warp_wait<kNsConv>(v_full, j & 1);
                    if (!ok) break;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        offs[(j & 1) * kKeysT + ht + 64 * i] = at[i];
                        key_scales[(j & 1) * kKeysT + ht + 64 * i] = two[i];
                    }
                    const uint32_t r = ranges_of(two[0], two[1]);
                    if (lane < 2) ranges[(j & 1) * 4 + (warp & 1) + 2 * lane] = r;
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(look_full + (j & 1));
                    place(j + 1);
                    entries(j + 2);
                    look(j + 2);
                }
                if (bad) report(a.dev_status, IDX_STATUS_BAD_PAGE);
            }
        }
        // Warp 0 issues the MMAs: it has nothing else to do meanwhile.
        const uint32_t base = tc::smem_u32(sm);
        // Round j: O += P V of step j and S of step j + 1, then the softmax of step j + 1.
        for (int j = -1; j < n && !idle; ++j) {
            if (warp == 0) {
                if (j >= 0) {
                    ok = warp_wait<kNsIssue>(v_full, j & 1) && warp_wait<kNsIssue>(p_full, j & 1);
                    if (ok) issue_outputs<D>(tm_o, tm_s, base + S::kV, j > 0, o_done);
                }
                if (ok && j + 1 < n) {
                    // P of step j lies where the next S goes: its product has to be done
                    ok = warp_wait<kNsIssue>(k_full, (j + 1) & 1) &&
                         warp_wait<kNsIssue>(j < 0 ? q_full : o_done, j < 0 ? 0 : j & 1);
                    if (ok) issue_scores<D>(tm_s, base + S::kQ, base + S::kK, s_full);
                }
            }
            if (!ok || j + 1 >= n) break;
            ok = warp_wait<kNsSoft>(s_full, (j + 1) & 1);
            if (!ok) break;
            tc::tc_fence_after();
            if constexpr (kSel) {
                if (scales[((j + 1) & 1) * kKeysT].w != 0.0f)
                    step_keyed(j + 1);
                else
                    step(j + 1, std::false_type{});
            } else {
                if (__any_sync(kFull, k0 + (j + 2) * kKeysT > vis))
                    step(j + 1, std::true_type{});
                else
                    step(j + 1, std::false_type{});
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(p_full);
        }
        if (warp == 0) {  // what was issued has to finish before the tensor memory is given back
            if (tc::elect_one()) tc::mma_commit(drain);
            __syncwarp();
            ok = warp_wait<kNsIssue>(drain, 0) && ok;
        }
        // ---- the row's result -------------------------------------------------------------------------
        // V's barrier too, long complete: it orders nan_key
        if (ok && n > 0 && !idle) ok = warp_wait<kNsSoft>(o_done, (n - 1) & 1) && warp_wait<kNsSoft>(v_full, (n - 1) & 1);
        if (ok && !idle) {
            tc::tc_fence_after();
            if (rc < 0.0f && l != 0.0f) l = __int_as_float(0x7fc00000);
            bool nan = !kSel && *nan_key < vis;
            if constexpr (kTree && !kSel)
                nan = nan_nodes[kTreeMaxNodes / 32] || tree_sees(mask, a.tree_words, s.nq, nan_nodes);
            store_rows<D, kHalf>(a, tm_o + lanes, sm + S::kK + warp * 32 * kOutRow<D>, n > 0, real, tok, hq, z, m, l, nan);
        }
    } else {
        // ---- converters --------------------------------------------------------------------------------
        const int ct = tid - 128, cw = ct >> 5;
        using C = ConvShare<D>;
        const C my(ct);
        constexpr int kPieces = C::kPieces;
        // keys that the tile's first row does not see though another does begin here
        const int vis_first = kSel ? 0 : kTree ? front : (int)visible_keys(s.len, s.nq, row0 / G, a.causal);
        uint4 rk[kPieces], rv[8];
        uint32_t my_scale = 0;  // the key's or block's two scale bytes, bit 16 set; 0: not to be used
        bool bad = false;

        // Lookups run ahead: a step's pages are loaded one step before its rows, and with a list (thread
        // ct looks after entry ct of a step) its entries two steps before.
        int32_t ent = -1, ent_n = -1;
        int32_t page[2] = {-1, -1};                     // the second: keys 64 .. of the step
        const uint8_t* rows_at[2] = {nullptr, nullptr};  // key 0 of the step, seen from either half
        int keys = 0;                                    // of the step
        auto lookup = [&](int j) {
            if constexpr (kSel) {
                page[0] = counts(j, ct, ent) ? pt[ent >> lp] : -1;
            } else {
                const int kt = k0 + j * kKeysT;
                page[0] = kt < k1 ? pt[kt >> lp] : -1;
                page[1] = kt + 64 < k1 ? pt[(kt + 64) >> lp] : -1;
            }
        };
        // A tree's context is read by few units, mostly once: its keys are sent for kFar steps ahead, from memory to L2, by two
        // threads (a page of 64 keys each); the loads into registers come one step ahead and would wait for memory.
        int32_t far_page = -1;  // of the step that is sent for next
        [[maybe_unused]] auto far_lookup = [&](int j) {
            if constexpr (kTree && !kSel) {
                const int key = k0 + j * kKeysT + ct;
                far_page = (ct & 63) == 0 && key < k1 ? pt[key >> lp] : -1;
            }
        };
        [[maybe_unused]] auto send_for = [&](int j) {
            if constexpr (kTree && !kSel) {
                const int key = k0 + j * kKeysT + ct;
                if ((uint32_t)far_page < (uint64_t)a.num_pages)
                    tc::bulk_prefetch(pool + (int64_t)far_page * a.page_stride + (int64_t)(key & (P - 1)) * 2 * D,
                                      min(64, k1 - key) * 2 * D);
            }
        };
        auto place = [&](int j) {
            my_scale = 0;
            if constexpr (kSel) {
                const bool seen = counts(j, ct, ent), in = (uint32_t)page[0] < (uint64_t)a.num_pages;
                int64_t at = -1;
                bad |= seen && !in;
                if (seen && in) {
                    const int tok = ent & (P - 1);
                    at = (int64_t)page[0] * a.page_stride;
                    my_scale = *reinterpret_cast<const uint16_t*>(pool + at + 2ll * P * D + 2 * (tok / kKvBlock)) | 65536u;
                    at += (int64_t)tok * 2 * D;
                }
                // the places of step j - 2 have been read: conv_all() came since
                offs[(j & 1) * kKeysT + ct] = at;
                conv_sync();
            } else {
                keys = k1 - (k0 + j * kKeysT);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool in = (uint32_t)page[h] < (uint64_t)a.num_pages;
                    bad |= !in && 64 * h < keys;
                    const uint8_t* at = pool + (int64_t)page[h] * a.page_stride;
                    // this thread's block of 16 keys
                    if (in && (ct & 15) == 0 && ct / 64 == h && ct < keys)
                        my_scale = *reinterpret_cast<const uint16_t*>(at + 2ll * P * D + 2 * ((ct & (P - 1)) / kKvBlock)) | 65536u;
                    rows_at[h] = in ? at - (h && P == 64 ? 64 * 2 * D : 0) : nullptr;
                }
            }
        };
        auto load_k = [&](int j) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int key = my.k_key + C::kKeyStep * i;
                const uint8_t* half = rows_at[2 * i / kPieces];
                const uint8_t* src = half + key * 2 * D;
                bool in = half != nullptr && key < keys;
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
                const uint8_t* half = cw >= 2 ? rows_at[1] : rows_at[0];
                const uint8_t* src = half + key * 2 * D;
                bool in = half != nullptr && key < keys;
                if constexpr (kSel) {
                    const int64_t at = offs[(j & 1) * kKeysT + key];
                    src = pool + at;
                    in = at >= 0;
                }
                uint4 w = make_uint4(0, 0, 0, 0);
                if constexpr (D == 128) {
                    if (in) w = *reinterpret_cast<const uint4*>(src + D + 16 * my.dg);
                } else {
                    uint2 y = make_uint2(0, 0);
                    if (in) y = *reinterpret_cast<const uint2*>(src + D + 8 * my.dg);
                    w.x = y.x;
                    w.y = y.y;
                }
                rv[i] = w;
            }
        };
        // A list's keys have scales of their own. Where a step's lie within 2^15 of one another and every key
        // counts, they are folded into the fp16 operands (exact: a code is at least 2^-9, fp16
        // reaches 2^-24) and the softmax sees one scale pair; otherwise it takes a pair per key.
        int k_top = 0, v_top = 0;  // largest scale bytes of the step
        bool fold = false;
        auto publish = [&](int j) {  // before the barrier
            const uint32_t r = ranges_of(my_scale, my_scale);
            key_scales[(j & 1) * kKeysT + ct] = my_scale;
            if (lane == 0) ranges[(j & 1) * 4 + cw] = r;
        };
        auto collect = [&](int j) {  // behind it
            const uint4 r = *reinterpret_cast<const uint4*>(ranges + (j & 1) * 4);
            const uint32_t hi = __vmaxu4(__vmaxu4(r.x, r.y), __vmaxu4(r.z, r.w));
            const uint32_t lo = __vminu4(__vminu4(r.x, r.y), __vminu4(r.z, r.w));
            k_top = hi & 255;
            v_top = hi >> 16 & 255;
            fold = k_top - (int)(lo >> 8 & 255) <= 15 && v_top - (int)(lo >> 24) <= 15;
        };
        auto down = [&](int by) -> uint32_t {  // 2^-by as fp16 bits, by in 0 .. 15
            return by < 15 ? (uint32_t)(15 - by) << 10 : 0x0200u;
        };
        auto write_k = [&](int j) {
            if (helped) my_scale = key_scales[(j & 1) * kKeysT + ct];
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
                write_k_piece<D>(sm + S::kK, rk[i], key, my.kp, f);
            }
            if constexpr (kSel) {
                if (!fold)
                    scales[(j & 1) * kKeysT + ct] = sc;
                else if (ct < 8)
                    scales[(j & 1) * kKeysT + ct] = make_float4(__uint_as_float((uint32_t)k_top << 23), (float)(v_top - 127),
                                                                ex2((float)(127 - v_top)), 0.0f);
            } else if ((ct & 15) == 0) {
                scales[(j & 1) * kKeysT + ct / 16] = sc;
            }
            tc::fence_proxy_async();
            tc::mbar_arrive(k_full);
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
            if constexpr (!kSel) {
                const int end = k0 + (j + 1) * kKeysT;
                if (end > vis_first && vis_first < kv_end) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        bool hit = clear_nan_codes(rv[i].x) | clear_nan_codes(rv[i].y);
                        if constexpr (D == 128) hit |= clear_nan_codes(rv[i].z) | clear_nan_codes(rv[i].w);
                        const int key = end - kKeysT + 8 * my.kg + i;
                        if constexpr (kTree) {
                            if (hit) atomicOr(&nan_nodes[key < front ? kTreeMaxNodes / 32 : (key - front) >> 5], 1u << ((key - front) & 31));
                        } else {
                            if (hit) atomicMin(nan_key, key);
                        }
                    }
                }
            }
            write_v_block<D>(sm + S::kV, rv, my.kg, my.dg, kSel && fold, f);
            tc::fence_proxy_async();
            tc::mbar_arrive(v_full);
        };

        if (n > 0) {
            if (!helped) {
                if constexpr (kSel) {
                    ent = load_entry(0, ct);
                    ent_n = load_entry(1, ct);
                }
                lookup(0);
                for (int j = 1; j < kFar; ++j) {
                    far_lookup(j);
                    send_for(j);
                }
                far_lookup(kFar);
            }
            // Round j: K of step j + 1 to shared memory (where step j's product has read), loads of step
            // j + 2's K; V of step j + 1 (where O += P V has read), loads of step j + 2's V.
#pragma unroll 1
            for (int j = -2; j + 1 < n; ++j) {
                if (j >= 0) ok = warp_wait<kNsConv>(s_full, j & 1) && ok;
                if constexpr (kSel) {
                    if (!helped) {
                        if (j >= -1) publish(j + 1);
                        ok = conv_all(ok);  // leave together: place() has a barrier
                    }
                    if (j >= -1) collect(j + 1);
                }
                if (!ok) break;
                if (j >= -1) write_k(j + 1);
                if (j + 2 < n) {
                    if (helped) {
                        ok = warp_wait<kNsConv>(look_full + (j & 1), (j + 2) >> 1 & 1);
                        if (!ok) break;
                    } else {
                        send_for(j + 2 + kFar);
                        far_lookup(j + 3 + kFar);
                        place(j + 2);
                    }
                    load_k(j + 2);
                    if (!helped) {
                        if constexpr (kSel) {
                            ent = ent_n;
                            ent_n = load_entry(j + 4, ct);
                        }
                        lookup(j + 3);
                    }
                }
                if (j >= 0) ok = warp_wait<kNsConv>(o_done, j & 1) && ok;
                if (j >= -1) write_v(j + 1);
                if (j + 2 < n) load_v(j + 2);
            }
        }
        if (bad) report(a.dev_status, IDX_STATUS_BAD_PAGE);
    }
    if (!ok) report(a.dev_status, IDX_STATUS_TIMEOUT);
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 0) tc::tmem_dealloc(tm_s, 256);
}

template <int D, bool kHalf, bool kSel, bool kTree>
cudaError_t launch_tile(const AttnArgs& a, cudaStream_t st) {
    constexpr int smem = SmemT<D>::kBytes;
    auto* kernel = attn_tile_kernel<D, kHalf, kSel, kTree>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(allowed, kernel, smem);
    if (e != cudaSuccess) return e;
    const int64_t units = kSel ? a.T * ((a.group + kRowsT - 1) / kRowsT)
                               : a.B * (((int64_t)a.max_q_len * a.group + kRowsT - 1) / kRowsT);
    return launch_pdl(kernel, dim3((unsigned)units, (unsigned)a.kv_heads, (unsigned)a.n_split), dim3(kThreadsT), smem, st,
                      a);
}

template <int D, bool kHalf>
cudaError_t launch_tile_d(const AttnArgs& a, cudaStream_t st) {
    if (a.tree) return a.sel ? launch_tile<D, kHalf, true, true>(a, st) : launch_tile<D, kHalf, false, true>(a, st);
    return a.sel ? launch_tile<D, kHalf, true, false>(a, st) : launch_tile<D, kHalf, false, false>(a, st);
}

}  // namespace

cudaError_t launch_attn_tile(const AttnArgs& a, cudaStream_t st) {
    if (a.head_dim == 128) return a.ftype == IDX_FP16 ? launch_tile_d<128, true>(a, st) : launch_tile_d<128, false>(a, st);
    return a.ftype == IDX_FP16 ? launch_tile_d<64, true>(a, st) : launch_tile_d<64, false>(a, st);
}

}  // namespace idx
