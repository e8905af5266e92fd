// attn.cu -- attention over the 8-bit paged KV cache for few query rows per kv head (decode), the join of a
// split key axis, and the choice between this kernel and the tensor-memory one (attn_tc.cu).
//
// A unit is up to 16 query rows of one kv head (the rows of its group of heads, token after
// token) against a range of keys. Its four warps take 32 keys in turn, each with a running softmax
// of its own; they are joined at the end. With 16 rows the work is streaming: 2*D bytes a key,
// 64*D multiply-adds. K and V go by cp.async (whole 128-byte lines: a quarter warp that touches more
// lines than one pays for each) into a ring of the warp's own in shared memory, a step in flight while one is
// worked on, and from there as fp16 (exact for e4m3) into mma.m16n8k16. Both products are free to
// permute their contraction axis, so a thread's operands are 16 consecutive bytes:
//   S = Q K^T: thread (r, c) = (lane / 4, lane % 4) holds key r's dims 64i + 16c .. + 15, the
//     B operand of four steps over dims; Q is laid out to match.
//   O = P V: S's accumulator is P's A operand as it stands: rows r, r + 8, keys 2c, 2c+1, 8+2c,
//     9+2c. The thread holds those four keys' dims r*D/8 .. and pairs their bytes by prmt;
//     column n of step j is dim n*D/8 + j, so a thread ends with D/4 consecutive dims of a row.
// Measured in replayed graphs (bf16): 64 sequences of 8192 keys, 64 heads over 8, D = 128: 181 us, 5.9 TB/s of cache,
// 88 % of the measured copy rate (236 us with lanes' pieces of 16 bytes scattered over lines); two of 131071
// keys, 32 heads over 4, D = 64: 32 us with the join, 4.2 TB/s; one of 256 keys, 8 heads over one: 6.5 us, 11 to 12 with
// the host's call. Eleven warps on an SM, each a chain of loads, 64 mma.sync, two shuffles, exponentials and 64
// mma.sync a step, do not hide all of it: DRAM 65 %, issue 40 % busy.
#include "attn.cuh"

namespace idx {

namespace {

constexpr int kWarps = 4;
constexpr int kStages = 2;
constexpr int kKeys = 32;  // of a warp's step

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes from global to shared memory; zeros when ok is false
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// A warp's ring: per stage 32 keys, their D bytes of K and of V in rows of 128 bytes (D = 128: K rows, then
// V rows; D = 64: K and V halves of one row). 16-byte chunk x of key t's row lies at chunk
// x ^ swizzle(t), which keeps both products' reads free of bank conflicts: 8 lanes read K chunks
// 4d .. 4d+3 of two neighbouring keys, or V chunks of two dims groups of keys 0, 2, 4, 6 apart.
template <int D>
struct Ring {
    static constexpr int kVB = D / 8;               // bytes of V per key and lane
    static constexpr int kVAt = D == 128 ? kKeys * 128 : 0;
    static constexpr int kStage = kKeys * 2 * D;
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kLd = D + 4;  // row of the join buffer
    static constexpr int kJoin = kWarps * 16 * kLd * 4;
    static constexpr int kBytes = kRing > kJoin ? kRing : kJoin;
};
__device__ __forceinline__ constexpr int swizzle(int t) { return (((t >> 1) & 3) << 1) ^ ((t & 1) << 2); }

// kDiag: rows of a unit may see unlike numbers of keys (dense, causal, several queries to a sequence). The ring starts on
// a 128-byte line: 16 bytes past one, 64 x 8192 keys took 205 us.
template <int D, bool kHalf, bool kSel, bool kDiag>
__global__ void __launch_bounds__(kWarps * 32, 3) attn_rows_kernel(const AttnArgs a) {
    using R = Ring<D>;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ float2 ml[kWarps][16];
    __shared__ int nan_key[kDiag ? kWarps : 1];  // lowest key whose V held a NaN code that was taken out
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
    pdl_wait();
    if (a.n_split > 1) pdl_launch_dependents();  // the join

    // ---- the unit: sequence, rows, keys --------------------------------------------------------
    const int G = a.group, head = blockIdx.y, z = blockIdx.z;
    int b, row0;           // first of the unit's rows: (token of the sequence) * G + head of the group
    int64_t tok0;          // query row that row 0 counts from
    int rows, kv_end;      // rows that exist; end of the keys (entries) that some row may see
    SeqRows s;
    if constexpr (kSel) {
        const int tiles = (G + 15) / 16;
        const int64_t t = blockIdx.x / tiles;
        b = warp_seq_of_query(a, t);
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
    const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    // copies: a lane takes 16-byte piece ci of key ck + i * kCopyKeys (a quarter warp: one 128-byte line)
    constexpr int kPieces = D / 8, kCopyKeys = 32 / kPieces, kCopies = kKeys / kCopyKeys;
    const int ci = lane % kPieces, ck = lane / kPieces;
    auto ring_at = [&](int t) -> uint32_t {  // where piece ci of key t goes
        return (D == 128 ? (ci >> 3) * R::kVAt : 0) + t * 128 + (((ci & 7) ^ swizzle(t)) << 4);
    };
    const int P = a.page_size, lp = P == 128 ? 7 : 6;
    const uint8_t* pool = a.pool + (int64_t)head * kv_head_bytes(P, D);
    const int32_t* pt = a.page_table + (int64_t)b * a.pt_stride;
    constexpr int kStep = kWarps * kKeys;
    const int kw = k0 + kKeys * warp;  // this warp's first key; its next ones are kStep further
    const int n_it = k1 > kw ? (k1 - kw + kStep - 1) / kStep : 0;
    const int vis_lo = __shfl_sync(kFull, vis[0], 0);  // rows see more and more keys: row 0 the fewest
    bool bad_page = false;

    // Lookups run ahead: a step's page is loaded one step before its copies are issued and, with a
    // list (lane l looks after entry l of the step), its entry two steps before.
    int32_t page = -1, ent = -1, ent_n = -1;
    auto load_entry = [&](int it) -> int32_t {
        const int e = kw + kStep * it + lane;
        return e < k1 ? a.sel[tok0 * a.sel_stride + e] : -1;
    };
    auto load_page = [&](int it) -> int32_t {
        if constexpr (kSel) return (ent >= 0 && ent < vis[0]) ? pt[ent >> lp] : -1;
        return it < n_it ? pt[(kw + kStep * it) >> lp] : -1;
    };
    // The scale bytes of a step, loaded with its copies. Dense: K, V of block 0, K, V of block 1, the same in
    // every lane. List: K, V of entry l's block, bit 16 set where the entry counts.
    uint32_t scales_n = 0;
    bool page_ok_n = false;
    auto issue = [&](int it) {
        const uint32_t at = (it & (kStages - 1)) * R::kStage;
        scales_n = 0;
        if constexpr (kSel) {
            const bool seen = ent >= 0 && ent < vis[0], in = (uint32_t)page < (uint64_t)a.num_pages;
            bad_page |= seen && !in;
            const int pg = seen && in ? page : -1, tok = ent & (P - 1);
            if (pg >= 0)
                scales_n = *reinterpret_cast<const uint16_t*>(pool + (int64_t)pg * a.page_stride + 2ll * P * D +
                                                             2 * (tok / kKvBlock)) | 65536u;
            const int64_t row = pg < 0 ? -1 : (int64_t)pg * a.page_stride + tok * 2 * D;
            const int lo = (int)row, hi = (int)(row >> 32);
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int t = ck + kCopyKeys * i;
                const uint32_t l = __shfl_sync(kFull, lo, t);
                const int h = __shfl_sync(kFull, hi, t);
                const int64_t from = (int64_t)(((uint64_t)(uint32_t)h << 32) | l);
                cp_async(ring_s + at + ring_at(t), pool + (h < 0 ? 0 : from + 16 * ci), h >= 0);
            }
        } else {
            const int kb = kw + kStep * it;
            page_ok_n = it < n_it && (uint32_t)page < (uint64_t)a.num_pages;
            bad_page |= it < n_it && !page_ok_n;
            if (page_ok_n) {
                const uint8_t* base = pool + (int64_t)page * a.page_stride;
                const int tok = kb & (P - 1);
                scales_n = *reinterpret_cast<const uint32_t*>(base + 2ll * P * D + 2 * (tok / kKvBlock));
                const uint8_t* row = base + tok * 2 * D;
                const uint8_t* src = row + ck * 2 * D + 16 * ci;
                auto copy = [&](auto whole_tag) {  // whole: no key of the step lies behind the end
                    constexpr bool kWhole = decltype(whole_tag)::value;
#pragma unroll
                    for (int i = 0; i < kCopies; ++i) {
                        const int t = ck + kCopyKeys * i;
                        cp_async(ring_s + at + ring_at(t), src + kCopyKeys * i * 2 * D, kWhole || kb + t < k1);
                    }
                };
                if (kb + kKeys <= k1)
                    copy(std::true_type{});
                else
                    copy(std::false_type{});
            }
        }
        cp_async_commit();
    };

    float m[2] = {neg_inf(), neg_inf()}, l[2] = {0.0f, 0.0f};
    float o[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[j][x] = 0.0f;

    // kMask: some key may not be visible to some row (the end of what a row sees; lists)
    auto compute = [&](int it, uint32_t scales, auto mask_tag) {
        [[maybe_unused]] constexpr bool kMask = decltype(mask_tag)::value;
        const uint8_t* sp = ring + (it & (kStages - 1)) * R::kStage;
        [[maybe_unused]] const int kb = kw + kStep * it;
        float sc[kKeys / 8][4];
#pragma unroll
        for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) sc[j][x] = 0.0f;
#pragma unroll
        for (int d = 0; d < D / 64; ++d)
#pragma unroll
            for (int j = 0; j < kKeys / 8; ++j) {
                const uint4 w = *reinterpret_cast<const uint4*>(sp + (8 * j + r) * 128 + (((4 * d + c) ^ swizzle(r)) << 4));
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t lo, hi;
                    e4m3x4_to_f16x4(u[x], lo, hi);
                    mma16816(sc[j], qa[d][x], lo, hi);
                }
            }
        // u = s * c + Ev; masked ones to -inf
        float ev[kKeys / 4], mx[2] = {neg_inf(), neg_inf()};
        [[maybe_unused]] uint32_t use = ~0u;  // bit k: the thread's key 8(k/2) + 2c + k%2 counts
#pragma unroll
        for (int k = 0; k < kKeys / 4; ++k) {
            uint32_t two;
            if constexpr (kSel) {
                two = __shfl_sync(kFull, scales, (k >> 1) * 8 + 2 * c + (k & 1));
                if (!(two >> 16)) use &= ~(1u << k);
            } else {
                two = k < 4 ? scales : scales >> 16;
            }
            const float kc = k_scale(two);
            ev[k] = v_exponent(two);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float& v = sc[k >> 1][2 * i + (k & 1)];
                v = fmaf(v, rc[i] * kc, ev[k]);
                if constexpr (kSel)
                    v = (use >> k) & 1u ? v : neg_inf();
                else if constexpr (kMask)
                    v = kb + (k >> 1) * 8 + 2 * c + (k & 1) < vis[i] ? v : neg_inf();
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
        uint32_t pa[kKeys / 16][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // a row that saw nothing yet: its weights are 2^-inf
            const float sub = m[i] == neg_inf() ? 0.0f : kShift - m[i];
#pragma unroll
            for (int h = 0; h < kKeys / 16; ++h) {
                float p[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) p[k] = ex2(sc[2 * h + (k >> 1)][2 * i + (k & 1)] + sub);
                if constexpr (kSel) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        l[i] = fmaf(p[k], (use >> (4 * h + k)) & 1u ? ex2(-ev[4 * h + k]) : 0.0f, l[i]);
                } else {
                    l[i] = fmaf((p[0] + p[1]) + (p[2] + p[3]), ex2(-ev[4 * h]), l[i]);
                }
                pa[h][i] = half2_bits(p[0], p[1]);
                pa[h][2 + i] = half2_bits(p[2], p[3]);
            }
        }
        // O += P V, 4 dims of four keys at a time
#pragma unroll
        for (int h = 0; h < kKeys / 16; ++h) {
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = 16 * h + (k >> 1) * 8 + 2 * c + (k & 1);
                if constexpr (D == 128) {
                    v[k] = *reinterpret_cast<const uint4*>(sp + R::kVAt + t * 128 + ((r ^ swizzle(t)) << 4));
                } else {
                    const uint2 w = *reinterpret_cast<const uint2*>(sp + t * 128 + (((4 + (r >> 1)) ^ swizzle(t)) << 4) + 8 * (r & 1));
                    v[k].x = w.x;
                    v[k].y = w.y;
                }
            }
#pragma unroll
            for (int y = 0; y < R::kVB / 4; ++y) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = y == 0 ? v[k].x : y == 1 ? v[k].y : y == 2 ? v[k].z : v[k].w;
                uint32_t b0[4], b1[4];
                e4m3x4_to_f16x4(__byte_perm(w[0], w[1], 0x5140), b0[0], b0[1]);
                e4m3x4_to_f16x4(__byte_perm(w[0], w[1], 0x7362), b0[2], b0[3]);
                e4m3x4_to_f16x4(__byte_perm(w[2], w[3], 0x5140), b1[0], b1[1]);
                e4m3x4_to_f16x4(__byte_perm(w[2], w[3], 0x7362), b1[2], b1[3]);
#pragma unroll
                for (int q = 0; q < 4; ++q) mma16816(o[4 * y + q], pa[h], b0[q], b1[q]);
            }
        }
    };

    // V's NaN codes taken out of a step's keys that some row does not see.
    [[maybe_unused]] auto clear_v = [&](int it) {
        constexpr int kVPieces = D / 16;
        uint8_t* sp = ring + (it & (kStages - 1)) * R::kStage + R::kVAt;
        const int kb = kw + kStep * it, t0 = max(vis_lo - kb, 0), t1 = min(k1 - kb, kKeys);
#pragma unroll 1
        for (int x = t0 * kVPieces + lane; x < t1 * kVPieces; x += 32) {
            const int t = x / kVPieces, chunk = x % kVPieces + (D == 128 ? 0 : kVPieces);
            uint4* at = reinterpret_cast<uint4*>(sp + t * 128 + ((chunk ^ swizzle(t)) << 4));
            uint4 w = *at;
            if (clear_nan_codes(w.x) | clear_nan_codes(w.y) | clear_nan_codes(w.z) | clear_nan_codes(w.w)) {
                *at = w;
                atomicMin(&nan_key[warp], kb + t);
            }
        }
        __syncwarp();
    };

    if (kDiag && lane == 0) nan_key[warp] = INT32_MAX;
    if (n_it > 0) {
        if constexpr (kSel) {
            ent = load_entry(0);
            ent_n = load_entry(1);
        }
        page = load_page(0);
        // A round: the copies of step it + 1 go out, the ones of step it have arrived.
        uint32_t scales = 0;
        bool page_ok = false;
        auto next = [&](int it) {
            scales = scales_n;
            page_ok = page_ok_n;
            __syncwarp();  // the stage that comes next has been read by every lane
            issue(it + 1);
            if constexpr (kSel) {
                ent = ent_n;
                ent_n = load_entry(it + 3);
            }
            page = load_page(it + 2);
            cp_async_wait<kStages - 1>();
            __syncwarp();  // every lane's copies have arrived
        };
        next(-1);
        if constexpr (kSel) {
#pragma unroll 1
            for (int it = 0; it < n_it; ++it) {
                next(it);
                compute(it, scales, std::true_type{});
            }
        } else {
            // A unit's rows see at most 15 keys more the one than the other, and a warp's steps are 128 keys
            // apart: only its last one can hold a key that some row does not see. Keys of a page outside the
            // pool do not exist.
#pragma unroll 1
            for (int it = 0; it < n_it - 1; ++it) {
                next(it);
                if (page_ok) compute(it, scales, std::false_type{});
            }
            next(n_it - 1);
            if (page_ok) {
                if constexpr (kDiag) clear_v(n_it - 1);
                compute(n_it - 1, scales, std::true_type{});
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
        if constexpr (kDiag) {
            int least = INT32_MAX;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) least = min(least, nan_key[w]);
            if (least < INT32_MAX && least < (int)visible_keys(s.len, s.nq, at / G, a.causal))
                v.x = v.y = v.z = v.w = __int_as_float(0x7fc00000);
        }
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

// Joins the splits of a key axis. A (query row, head) is joined by kPerRow of a CTA's four warps: all four
// take splits in turn where rows are few, so that their loads are in flight together, and sum in
// shared memory (64 rows of 38 splits: 32 us with the attention against 39); enough rows to fill the GPU
// take a warp each (4096 rows of 4 splits: 180 against 182 us with the attention, 32768 of 2: 56 against 78).
// The call's last kernel, this one or a sole attention kernel, lets nothing start beside it: out may be what the
// next call reads before its wait (q or k of the pre-processing).
constexpr int kJoinWarps = 4;
constexpr int kJoinAlone = 8;  // rows per SM from which a warp joins one
template <int D, bool kHalf, int kPerRow>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_join_kernel(const AttnArgs a) {
    constexpr int kDims = D / 32;  // dims of a lane
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = warp % kPerRow;
    const int64_t step = a.T * a.q_heads;
    const int64_t row = (int64_t)blockIdx.x * (kJoinWarps / kPerRow) + warp / kPerRow, t = row / a.q_heads;
    const int hq = (int)(row % a.q_heads);
    pdl_wait();
    if (row >= step) return;  // a whole warp, with kPerRow = kJoinWarps never
    const int b = warp_seq_of_query(a, t);
    if (b < 0 || seq_rows(a, b).nq < 0) return;  // the same for all warps of a row
    // every warp: all maxima, two splits to a lane at most
    float2 ml[2];
    float M = neg_inf();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        ml[i] = lane + 32 * i < a.n_split ? a.part_ml[row + (lane + 32 * i) * step] : make_float2(neg_inf(), 0.0f);
        M = fmaxf(M, ml[i].x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    float g[2], L = 0.0f, v[kDims];
#pragma unroll
    for (int i = 0; i < 2; ++i) g[i] = ml[i].x == M ? 1.0f : ex2(ml[i].x - M);
#pragma unroll
    for (int i = 0; i < kDims; ++i) v[i] = 0.0f;
#pragma unroll 4
    for (int z = first; z < a.n_split; z += kPerRow) {
        const float gz = __shfl_sync(kFull, z < 32 ? g[0] : g[1], z & 31);
        const float lz = __shfl_sync(kFull, z < 32 ? ml[0].y : ml[1].y, z & 31);
        if (lz == 0.0f) continue;  // that split had no key for this row and wrote no O
        L = fmaf(gz, lz, L);
        const float* src = a.part_o + (row + z * step) * D + kDims * lane;
        float x[kDims];
        if constexpr (kDims == 4)
            *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(src);
        else
            *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(src);
#pragma unroll
        for (int i = 0; i < kDims; ++i) v[i] = fmaf(gz, x[i], v[i]);
    }
    if constexpr (kPerRow > 1) {
        __shared__ float part[kJoinWarps][D];
        __shared__ float part_l[kJoinWarps];
#pragma unroll
        for (int i = 0; i < kDims; ++i) part[warp][kDims * lane + i] = v[i];
        if (lane == 0) part_l[warp] = L;
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int w = 1; w < kJoinWarps; ++w) {
            L += part_l[w];
#pragma unroll
            for (int i = 0; i < kDims; ++i) v[i] += part[w][kDims * lane + i];
        }
    }
    const float n = L == 0.0f ? 0.0f : 1.0f / L;
    uint32_t* out = reinterpret_cast<uint32_t*>(a.out + t * a.out_row_stride + (int64_t)hq * a.out_head_stride) +
                    kDims / 2 * lane;
#pragma unroll
    for (int i = 0; i < kDims / 2; ++i) out[i] = store_pair<kHalf>(v[2 * i] * n, v[2 * i + 1] * n);
    if (a.lse && first == 0 && lane == 0) a.lse[row] = lse_of(M, L);
}

template <int D, bool kHalf, int kPerRow>
cudaError_t launch_join(const AttnArgs& a, cudaStream_t st) {
    constexpr int rows = kJoinWarps / kPerRow;
    const int64_t ctas = (a.T * a.q_heads + rows - 1) / rows;
    return launch_pdl(attn_join_kernel<D, kHalf, kPerRow>, dim3((unsigned)ctas), dim3(kJoinWarps * 32), 0, st, a);
}

// Rows that share their keys: those of a sequence and a kv head, or with a list those of a query's group.
int64_t shared_rows(const AttnArgs& a) { return a.n_sel ? a.group : (int64_t)a.max_q_len * a.group; }

// Which kernel. Dense: up to two mma.sync tiles of shared rows this file's (32 heads over one kv head, 3000 keys of
// one sequence: 10.1 us against 14.8; 64 x 8192 keys: 59 against 58), more the tensor-memory one (64 heads, 64 x 8192
// keys: 62 against 93). Lists, whose keys are gathered for each tile: up to one (4096 queries x 1024 keys, 16 heads:
// 207 us against 380; 32 heads in two tiles 413 against 389).
struct Choice {
    bool tile;
    int64_t units;
    int per_sm;  // resident CTAs
};
Choice choose(const AttnArgs& a) {
    const int64_t rows = shared_rows(a), times = (a.n_sel ? a.T : (int64_t)a.B) * a.kv_heads;
    if (rows <= (a.n_sel ? 16 : 32)) return {false, times * ((rows + 15) / 16), 3};
    return {true, times * ((rows + 127) / 128), 2};
}

template <int D, bool kHalf, bool kSel, bool kDiag>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t st) {
    constexpr int smem = Ring<D>::kBytes;
    auto* kernel = attn_rows_kernel<D, kHalf, kSel, kDiag>;
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
    cudaError_t e = choose(a).tile                   ? launch_attn_tile(a, st)
                    : a.sel                          ? launch_rows<D, kHalf, true, false>(a, st)
                    : a.causal && a.max_q_len > 1    ? launch_rows<D, kHalf, false, true>(a, st)
                                                     : launch_rows<D, kHalf, false, false>(a, st);
    if (e != cudaSuccess || a.n_split <= 1) return e;
    const int64_t many = (int64_t)kJoinAlone * device_sm_count();
    return a.T * a.q_heads < many ? launch_join<D, kHalf, kJoinWarps>(a, st) : launch_join<D, kHalf, 1>(a, st);
}

}  // namespace

int64_t attn_plan(AttnArgs& a, int64_t bytes) {
    const int sms = device_sm_count();
    if (sms <= 0) return -1;
    const Choice choice = choose(a);
    const int64_t units = choice.units;
    const int64_t keys = a.n_sel ? a.n_sel : a.max_seq_len_k;
    const int64_t per_split = a.T * a.q_heads * (a.head_dim + 2) * 4;
    // Splits. Units that fill the resident CTAs (three or two to an SM) by themselves are cut until there are
    // about four rounds of them, in pieces of 1024 keys at least (64 sequences of 8192 keys, 8
    // kv heads: 205 / 180 / 180 / 186 us with 1 / 2 / 4 / 7 splits); fewer units are cut until they fill one
    // round, in pieces of 512 keys at least (two sequences of 131071 keys, 4 kv heads: 35 / 32 / 32
    // / 44 us with 32 / 38 / 57 / 64, the last one round and a bit), or of 256 where those are fewer
    // than the SMs (one sequence of 4000 keys: 20.3 / 13.9 / 10.4 / 8.9 us with 2 / 4 / 8 / 16).
    // The tensor-memory kernel's units hold up to 128 rows, whose partial results cost more than a
    // second round: they are cut to fill one (64 x 8192 keys, 64 heads over 1: 75 / 73 / 62 / 72 us with 2 /
    // 3 / 4 / 8; 512 queries on 8192 keys: 124 / 99 / 112 with 1 / 2 / 4) and not at all where
    // they do by themselves (prompts of 1024 and 2048: 34 and 80 us whole, 56 and 114 in 2). max_q_len only
    // bounds the number of queries, so the units that have rows are counted from T; where chunks are
    // uneven they are cut to fill three rounds (8 of 3 to 301 queries on up to 3300 keys: 48 / 31 / 27 /
    // 24 / 29 us with 1 / 2 / 4 / 6 / 8; no other batch of uneven chunks was measured).
    const int64_t slots = (int64_t)sms * choice.per_sm;
    int64_t want = 1;
    if (units > 0) {
        const auto least = [](int64_t x, int64_t y) { return x < y ? x : y; };
        const int64_t one_round_keys = units * keys <= 256ll * sms ? 256 : 512;
        if (choice.tile) {
            const int64_t filled = a.n_sel ? units : least(units, (a.T * a.group / 128 + a.B) * a.kv_heads);
            const bool uneven = !a.n_sel && 4 * a.T < 3ll * a.B * a.max_q_len;
            want = least(64, least((uneven ? 3 : 1) * slots / filled, keys / one_round_keys));
        } else {
            want = least(64, least(4 * slots / units, keys / 1024));
            if (units * want < slots + slots / 2) want = least(64, least(slots / units, keys / one_round_keys));
        }
        if (want < 1) want = 1;
    }
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
