// rope.cu - norms of queries and keys for each head with the position rotation in the same pass, its
// gradient, and the writes of keys and values to a paged cache of 16 or 4 bits with both on the way.
//
// A row x of D values becomes rot(n w), n = x / sqrt(mean(x^2) + eps): pair (a, b) of the first R columns
// turns to (a c - b s, b c + a s).  Every row is read and written once and carries a few operations a byte,
// so the time is that of the bytes (4 D a row forwards, 6 D backwards), or of the launch.
//
// A row is held by D / 16 lanes in two 16-byte pieces each, chosen so that a lane has both halves of its
// pairs: nothing but the sums crosses lanes.  A warp takes consecutive steps of 512 / D rows, a token's heads after
// one another, so that the token's angles are loaded once into registers (for each row, they would be twice the
// row's bytes).  Rows come through a ring in shared memory, several steps ahead (cp.async, each lane its own pieces,
// so that no lane waits for another): plain loads ahead would take the registers that the arithmetic needs.
#include "rows16.cuh"
#include "serving.h"

namespace gsr {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kCtasAnSm = 3, kBwdCtasAnSm = 2;

// What a lane holds of a row: 16-byte pieces c0 and c1, neighbouring lanes' next to each other (a warp's access then
// covers whole sectors; with both of a lane's pieces next to each other a plain copy took 44 us for 26).
struct LanePart {
    int c0, c1;
    bool t0, t1;                 // interleaved: whether a piece's pairs turn; else (t0) whether they turn with each other
};
template <int LANES>
__device__ __forceinline__ LanePart lane_part(int l, int R, bool interleaved) {
    const int rc = R >> 4;                       // lanes that hold pairs (i, i + R / 2)
    if (interleaved) return {l, l + LANES, 8 * l < R, 8 * (l + LANES) < R};
    if (l < rc) return {l, l + rc, true, true};
    return {l + rc, l + LANES, false, false};
}

// EXACT: each product and sum rounded by itself, so that codes of 4 bits do not hang on a contraction.
template <bool EXACT>
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float x = EXACT ? __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)) : fmaf(a, c, -b * s);
    b = EXACT ? __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)) : fmaf(b, c, a * s);
    a = x;
}
struct Angles {
    float c[8], s[8];
};
// A lane's angles of position pos; BACK: turned the other way.
template <bool BACK, int LANES>
__device__ __forceinline__ void load_angles(Angles& a, const float* table, long long pos, int R, bool interleaved, const LanePart& at, int l) {
    const float* row = table + pos * R;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (!(i ? at.t1 : at.t0)) continue;
        const float* c = row + (interleaved ? 4 * (l + i * LANES) : 8 * l + 4 * i);
        const float4 x = __ldg(reinterpret_cast<const float4*>(c)), y = __ldg(reinterpret_cast<const float4*>(c + R / 2));
        const float sign = BACK ? -1.0f : 1.0f;
        a.c[4 * i] = x.x; a.c[4 * i + 1] = x.y; a.c[4 * i + 2] = x.z; a.c[4 * i + 3] = x.w;
        a.s[4 * i] = sign * y.x; a.s[4 * i + 1] = sign * y.y; a.s[4 * i + 2] = sign * y.z; a.s[4 * i + 3] = sign * y.w;
    }
}
// v[0..7] is piece c0, v[8..15] piece c1.
template <bool EXACT>
__device__ __forceinline__ void rotate(float (&v)[16], const Angles& a, bool interleaved, const LanePart& at) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < 4 ? at.t0 : at.t1) turn<EXACT>(v[2 * i], v[2 * i + 1], a.c[i], a.s[i]);
    } else if (at.t0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn<EXACT>(v[i], v[8 + i], a.c[i], a.s[i]);
    }
}
// The angles of one token after another, for lanes that turn pairs.
struct TokenAngles {
    Angles angles;
    int token = -1, pos = 0, next_pos = 0;
    bool known = true;                  // the position is in the table
    template <bool BACK, int LANES>
    __device__ __forceinline__ void move(const RopeParams& p, int now, int s, int tokens, const LanePart& at, int l) {
        if (now == token || !p.table) return;
        if (p.positions) {
            pos = now == token + 1 && token >= 0 ? next_pos : __ldg(p.positions + now);
            next_pos = now + 1 < tokens ? __ldg(p.positions + now + 1) : 0;
        } else {
            pos = s;
        }
        token = now;
        known = pos >= 0 && pos < p.rows;
        if (known) load_angles<BACK, LANES>(angles, p.table, pos, p.R, p.interleaved, at, l);
    }
};
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
// A piece of 16 bytes to the ring, and waits for all but the last N steps' pieces of this lane.
__device__ __forceinline__ void copy_piece(uint4* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void commit_pieces() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_pieces() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Steps are counted through the tokens: `blocks` of them a token.
struct Cursor {
    int left, token, b, s, block;       // steps left; the token, its batch row and place; the step in the token
    __device__ __forceinline__ Cursor(int first, int count, const Divider& by_token, const Divider& by_seq) {
        left = count;
        token = by_token(first);
        block = first - token * (int)by_token.d;
        b = by_seq(token);
        s = token - b * (int)by_seq.d;
    }
    __device__ __forceinline__ void step(int blocks, int S) {
        --left;
        if (++block < blocks) return;
        block = 0;
        ++token;
        if (++s == S) {
            s = 0;
            ++b;
        }
    }
};
// Steps [first, first + count) of `units` for warp w of `warps`.
__device__ __forceinline__ void share_of(int units, int w, int warps, int& first, int& count) {
    const int each = (units + warps - 1) / warps;
    first = min((long long)w * each, (long long)units);
    count = min(each, units - first);
}
template <class T>
__device__ __forceinline__ void load_weight(const T* w, const LanePart& at, float (&to)[16]) {
    unpack8<T>(__ldg(reinterpret_cast<const uint4*>(w) + at.c0), to);
    unpack8<T>(__ldg(reinterpret_cast<const uint4*>(w) + at.c1), to + 8);
}
template <class T>
__device__ __forceinline__ void store_part(T* row, const LanePart& at, const float (&v)[16]) {
    reinterpret_cast<uint4*>(row)[at.c0] = pack8<T>(v);
    reinterpret_cast<uint4*>(row)[at.c1] = pack8<T>(v + 8);
}

// ---------------------------------------------------------------------------
// Forward, and the cache writes
// ---------------------------------------------------------------------------
// Of three values; the larger is NaN where one of them is.
__device__ __forceinline__ float min3(float a, float b, float c) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

enum Sink : int { kSinkRows, kSinkCache16, kSinkCache4 };

constexpr int kStages = 4;

// A token's steps: those of Q's heads, then K's, then (cache writes) V's.
struct RopePlan {
    Divider by_token, by_seq, by_page;
    int q_blocks, k_blocks, units;
};

// A row of 4 bits: per 64 values minimum m and scale s = (maximum - m) / 15, both rounded to T, and codes
// rint((x - m) / s) cut to 0..15.  A group that holds infinities or NaN, or spans more than a float, is NaN as a whole.
template <class T, int D>
__device__ __forceinline__ void store_row4(const Cache4& cache, long long page, int row, int head, const LanePart& at, int l,
                                           bool live, const float (&v)[16]) {
    constexpr int LANES = D / 16;
    uint32_t words[2] = {0u, 0u}, pair[D / 64];
    float m[D / 64], s[D / 64], low[2], high[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float* x = v + 8 * k;
        low[k] = min3(min3(x[0], x[1], x[2]), min3(x[3], x[4], x[5]), fminf(x[6], x[7]));
        high[k] = max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), max3(x[6], x[7], x[7]));
    }
    const int g0 = D > 64 ? at.c0 >> 3 : 0, g1 = D > 64 ? at.c1 >> 3 : 0;
#pragma unroll
    for (int g = 0; g < D / 64; ++g) {
        float lo = fminf(g0 == g ? low[0] : INFINITY, g1 == g ? low[1] : INFINITY);
        float hi = max3(g0 == g ? high[0] : -INFINITY, g1 == g ? high[1] : -INFINITY, -INFINITY);
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            const float other = __shfl_xor_sync(0xffffffffu, hi, o);
            hi = max3(hi, other, other);
        }
        const float span = hi - lo;                        // NaN, or infinite, with what is not finite
        const bool fine = span <= 3.402823466e38f;
        pair[g] = Pair<T>::pack(fine ? __fmul_rn(span, 1.0f / 15.0f) : NAN, fine ? lo : NAN);
        const float2 held = Pair<T>::unpack(pair[g]);
        s[g] = held.x;
        m[g] = held.y;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int g = k ? g1 : g0;
        const float sk = D > 64 && g ? s[D / 64 - 1] : s[0], mk = D > 64 && g ? m[D / 64 - 1] : m[0];
        if (sk > 0.0f) {
            // x / s as 15 times what a saturated product leaves in 0..1, off by at most 2^-18: divided only next to a
            // border.  A sum with 1.5 2^23 rounds to the nearest even and leaves the integer in its low bits
            // (conversions run at an eighth of the rate).
            constexpr uint32_t MAGIC = 0x4b400000u;
            const float magic = __uint_as_float(MAGIC), inv = __fdividef(1.0f, 15.0f * sk);
            float off = sk > 1e-30f && sk < 1e30f ? 0.0f : 1.0f;      // next to the type's ends 1 / s is not good enough
            uint32_t w = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = __saturatef((v[8 * k + i] - mk) * inv), c = fmaf(x, 15.0f, magic);
                off = fmaxf(off, fabsf(fmaf(x, 15.0f, magic - c)));
                w += (__float_as_uint(c) - MAGIC) * (1u << (4 * i));
            }
            if (!(off <= 0.49999f)) {
                w = 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w |= (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(v[8 * k + i] - mk, sk)), 0.0f), 15.0f) << (4 * i);
            }
            words[k] = w;
        }
    }
    if (!live) return;
    char* codes = cache.codes.data + page * cache.codes.page + (long long)row * cache.codes.row + head * cache.codes.head;
    reinterpret_cast<uint32_t*>(codes)[at.c0] = words[0];
    reinterpret_cast<uint32_t*>(codes)[at.c1] = words[1];
    if (l < D / 64) {
        char* params = cache.params.data + page * cache.params.page + (long long)row * cache.params.row + head * cache.params.head;
        reinterpret_cast<uint32_t*>(params)[l] = l ? pair[D / 64 - 1] : pair[0];
    }
}

template <class T, int D, int SINK>
__global__ void __launch_bounds__(kThreads, kCtasAnSm) gsr_rope_kernel(const __grid_constant__ RopeAppendParams a,
                                                                       const __grid_constant__ RopePlan plan) {
    constexpr int LANES = D / 16, ROWS = 32 / LANES;
    __shared__ uint4 ring[kWarps][kStages][2][32];
    const RopeParams& p = a.f;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LANES;
    const int blocks = (int)plan.by_token.d, tokens = p.B * p.S;
    int first, count;
    share_of(plan.units, blockIdx.x * kWarps + warp, gridDim.x * kWarps, first, count);
    if (count <= 0) return;
    const LanePart at_qk = lane_part<LANES>(l, p.table ? p.R : 0, p.interleaved), at_v = lane_part<LANES>(l, 0, false);

    struct Place {                       // which rows a step has
        bool is_q, is_v, live;
        int h;
    };
    auto place = [&](const Cursor& c) {
        Place x;
        x.is_q = c.block < plan.q_blocks;
        x.is_v = SINK != kSinkRows && c.block >= plan.q_blocks + plan.k_blocks;
        x.h = (c.block - (x.is_q ? 0 : x.is_v ? plan.q_blocks + plan.k_blocks : plan.q_blocks)) * ROWS + lane / LANES;
        x.live = x.h < (x.is_q ? p.Hq : p.Hkv);
        return x;
    };
    Cursor ahead(first, count, plan.by_token, plan.by_seq), now = ahead;
    int stage_ahead = 0, stage = 0;
    auto load = [&]() {
        if (ahead.left > 0) {
            const Place x = place(ahead);
            const Strided& src = x.is_q ? p.Q : x.is_v ? a.V : p.K;
            const LanePart& at = x.is_v ? at_v : at_qk;
            const uint4* from = reinterpret_cast<const uint4*>(static_cast<const T*>(src.data) + ahead.b * src.batch + ahead.s * src.row + x.h * src.head);
            if (x.live) {
                copy_piece(&ring[warp][stage_ahead][0][lane], from + at.c0);
                copy_piece(&ring[warp][stage_ahead][1][lane], from + at.c1);
            }
            ahead.step(blocks, p.S);
            stage_ahead = (stage_ahead + 1) % kStages;
        }
        commit_pieces();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) load();

    TokenAngles turned;
    int slot_token = -1, slot = -1;
#pragma unroll 1
    for (; now.left > 0; now.step(blocks, p.S)) {
        load();
        turned.template move<false, LANES>(p, now.token, now.s, tokens, at_qk, l);
        const Place x = place(now);
        const LanePart& at = x.is_v ? at_v : at_qk;
        const T* w = static_cast<const T*>(x.is_q ? p.q_weight : x.is_v ? nullptr : p.k_weight);
        const bool to_cache = SINK != kSinkRows && !x.is_q;
        if (to_cache && slot_token != now.token) {
            slot_token = now.token;
            slot = __ldg(a.slots + now.token);
            if (slot >= (long long)a.num_pages * a.page || (p.table && turned.pos < 0)) slot = -1;
        }
        wait_pieces<kStages - 1>();
        float v[16];
        uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
        if (x.live) {
            lo = ring[warp][stage][0][lane];
            hi = ring[warp][stage][1][lane];
        }
        stage = (stage + 1) % kStages;
        if (to_cache && slot < 0) continue;                // padding
        unpack8<T>(lo, v);
        unpack8<T>(hi, v + 8);
        if (w) {
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < 16; ++k) sum = fmaf(v[k], v[k], sum);
            const float r = rsqrtf(row_sum<LANES>(sum) * (1.0f / D) + p.eps);
            float weight[16];
            load_weight(w, at, weight);
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = v[k] * r * weight[k];
        }
        if (turned.known && !x.is_v) rotate<SINK == kSinkCache4>(v, turned.angles, p.interleaved, at);
        if (!turned.known && !x.is_v) {
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = turned.pos < 0 ? 0.0f : NAN;
        }
        if (!to_cache) {
            const Strided& to = x.is_q ? p.Qo : p.Ko;
            if (x.live) store_part(static_cast<T*>(to.data) + now.b * to.batch + now.s * to.row + x.h * to.head, at, v);
        } else {
            const long long page = plan.by_page(slot);
            const int row = slot - (int)page * a.page;
            if (SINK == kSinkCache16) {
                const Strided& to = x.is_v ? a.Vc : a.Kc;
                if (x.live) store_part(static_cast<T*>(to.data) + page * to.batch + row * to.row + x.h * to.head, at, v);
            } else {
                store_row4<T, D>(x.is_v ? a.V4 : a.K4, page, row, x.h, at, l, x.live, v);
            }
        }
    }
}

// CTAs of `units` steps: what fits on the SMs at once, or a step a warp.
int rope_ctas(long long units, int at_once) {
    const long long ctas = (units + kWarps - 1) / kWarps;
    return (int)(ctas < at_once ? ctas : at_once);
}

template <class T, int D, int SINK>
cudaError_t launch_rope(const RopeAppendParams& a, int sms, cudaStream_t stream) {
    const RopeParams& p = a.f;
    constexpr int ROWS = 512 / D;
    RopePlan plan{Divider(1), Divider((uint32_t)p.S), Divider((uint32_t)(a.page > 0 ? a.page : 1)), 0, 0, 0};
    plan.q_blocks = (p.Hq + ROWS - 1) / ROWS;
    plan.k_blocks = (p.Hkv + ROWS - 1) / ROWS;
    const int blocks = plan.q_blocks + (SINK == kSinkRows ? 1 : 2) * plan.k_blocks;
    plan.by_token = Divider((uint32_t)blocks);
    plan.units = (int)((long long)p.B * p.S * blocks);
    gsr_rope_kernel<T, D, SINK><<<(unsigned)rope_ctas(plan.units, kCtasAnSm * sms), kThreads, 0, stream>>>(a, plan);
    return cudaGetLastError();
}
template <int SINK>
cudaError_t launch_rope_type(const RopeAppendParams& a, bool bf16, int sms, cudaStream_t stream) {
    if (a.f.D == 64)
        return bf16 ? launch_rope<__nv_bfloat16, 64, SINK>(a, sms, stream) : launch_rope<__half, 64, SINK>(a, sms, stream);
    return bf16 ? launch_rope<__nv_bfloat16, 128, SINK>(a, sms, stream) : launch_rope<__half, 128, SINK>(a, sms, stream);
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------
// With dy the incoming gradient turned back, n = x r, dn = dy w:
//   dw = sum over rows of dy n,   dx = r (dn - n mean(dn n)) = r dn - x r^3 sum(dn x) / D.
// r is computed again from x, which has to be read anyway, so the forward pass stores nothing.  A CTA sums dw
// over its rows in registers (fp32, a lane's 16 columns), then over its warps; a second launch adds the CTAs'
// sums in their order, so that results repeat.
constexpr int kBwdStages = 3;

struct RopeBwdPlan {
    Divider by_q, by_k, by_seq;
    int q_units, k_units;
};

template <class T, int D>
__global__ void __launch_bounds__(kThreads, kBwdCtasAnSm) gsr_rope_bwd_kernel(const __grid_constant__ RopeBwdParams a,
                                                                           const __grid_constant__ RopeBwdPlan plan) {
    constexpr int LANES = D / 16, ROWS = 32 / LANES;
    __shared__ uint4 ring[kWarps][kBwdStages][4][32];
    float* const sums = reinterpret_cast<float*>(ring);    // of the warps, after the rows: D each
    const RopeParams& p = a.f;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LANES, tokens = p.B * p.S;
    const LanePart at = lane_part<LANES>(l, p.table ? p.R : 0, p.interleaved);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
        const Strided &G = part ? p.Ko : p.Qo, &X = part ? p.K : p.Q, &dX = part ? a.dK : a.dQ;
        const T* w = static_cast<const T*>(part ? p.k_weight : p.q_weight);
        const int heads = part ? p.Hkv : p.Hq;
        const Divider& by = part ? plan.by_k : plan.by_q;
        const int blocks = (int)by.d;
        float dw[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) dw[k] = 0.0f;
        int first, count;
        share_of(part ? plan.k_units : plan.q_units, blockIdx.x * kWarps + warp, gridDim.x * kWarps, first, count);
        Cursor ahead(first, count, by, plan.by_seq), now = ahead;
        int stage_ahead = 0, stage = 0;
        auto load = [&]() {
            if (ahead.left > 0) {
                const int h = ahead.block * ROWS + lane / LANES;
                if (h < heads) {
                    const uint4* g = reinterpret_cast<const uint4*>(static_cast<const T*>(G.data) + ahead.b * G.batch + ahead.s * G.row + h * G.head);
                    copy_piece(&ring[warp][stage_ahead][0][lane], g + at.c0);
                    copy_piece(&ring[warp][stage_ahead][1][lane], g + at.c1);
                    if (w) {
                        const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(X.data) + ahead.b * X.batch + ahead.s * X.row + h * X.head);
                        copy_piece(&ring[warp][stage_ahead][2][lane], x + at.c0);
                        copy_piece(&ring[warp][stage_ahead][3][lane], x + at.c1);
                    }
                }
                ahead.step(blocks, p.S);
                stage_ahead = stage_ahead == kBwdStages - 1 ? 0 : stage_ahead + 1;
            }
            commit_pieces();
        };
#pragma unroll
        for (int i = 0; i < kBwdStages - 1; ++i) load();
        TokenAngles turned;
#pragma unroll 1
        for (; now.left > 0; now.step(blocks, p.S)) {
            load();
            turned.template move<true, LANES>(p, now.token, now.s, tokens, at, l);
            const int h = now.block * ROWS + lane / LANES;
            const bool live = h < heads, counts = live && (!p.table || turned.pos >= 0);
            wait_pieces<kBwdStages - 1>();
            uint4 raw[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                raw[k] = make_uint4(0u, 0u, 0u, 0u);
                if (live && (k < 2 || w)) raw[k] = ring[warp][stage][k][lane];
            }
            stage = stage == kBwdStages - 1 ? 0 : stage + 1;
            float dy[16];
            unpack8<T>(raw[0], dy);
            unpack8<T>(raw[1], dy + 8);
            if (turned.known) rotate<false>(dy, turned.angles, p.interleaved, at);
            if (!turned.known) {
#pragma unroll
                for (int k = 0; k < 16; ++k) dy[k] = counts ? NAN : 0.0f;
            }
            if (w) {
                float v[16], weight[16];
                unpack8<T>(raw[2], v);
                unpack8<T>(raw[3], v + 8);
                load_weight(w, at, weight);
                float square = 0.0f, dot = 0.0f;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    square = fmaf(v[k], v[k], square);
                    weight[k] *= dy[k];
                    dot = fmaf(weight[k], v[k], dot);
                }
                const float r = rsqrtf(row_sum<LANES>(square) * (1.0f / D) + p.eps);
                const float back = row_sum<LANES>(dot) * (1.0f / D) * r * r * r;
                if (counts) {                              // padding adds nothing, whatever it holds
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        dw[k] = fmaf(dy[k] * v[k], r, dw[k]);
                        dy[k] = r * weight[k] - v[k] * back;
                    }
                }
            }
            if (!counts) {
#pragma unroll
                for (int k = 0; k < 16; ++k) dy[k] = 0.0f;
            }
            if (live) store_part(static_cast<T*>(dX.data) + now.b * dX.batch + now.s * dX.row + h * dX.head, at, dy);
        }
        wait_pieces<0>();
        if (!w) continue;
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int o = LANES; o < 32; o <<= 1) dw[k] += __shfl_xor_sync(0xffffffffu, dw[k], o);
        __syncthreads();
        if (lane < LANES) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sums[warp * D + 8 * at.c0 + k] = dw[k];
                sums[warp * D + 8 * at.c1 + k] = dw[8 + k];
            }
        }
        __syncthreads();
        if (threadIdx.x < D) {
            float t = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) t += sums[k * D + threadIdx.x];
            a.parts[((long long)part * a.ctas + blockIdx.x) * D + threadIdx.x] = t;
        }
        __syncthreads();
    }
}

// dw = sum of the CTAs' parts, a CTA for 32 columns: 32 lanes of rows, each in ascending order.
__global__ void __launch_bounds__(1024) gsr_rope_weights_kernel(const float* parts, int ctas, int D, float* dq_weight, float* dk_weight) {
    __shared__ float sums[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");     // launched while the rows' CTAs run
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
    float* to = blockIdx.y ? dk_weight : dq_weight;
    if (!to) return;
    float t = 0.0f;
#pragma unroll 8
    for (int i = y; i < ctas; i += 32) t += parts[((long long)blockIdx.y * ctas + i) * D + col];
    sums[y][threadIdx.x & 31] = t;
    __syncthreads();
    if (y == 0) {
        t = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += sums[i][threadIdx.x];
        to[col] = t;
    }
}

template <class T, int D>
cudaError_t launch_bwd(const RopeBwdParams& a, cudaStream_t stream) {
    const RopeParams& p = a.f;
    const long long tokens = (long long)p.B * p.S;
    cudaError_t e = cudaSuccess;
    if (a.ctas > 0) {
        RopeBwdPlan plan{Divider(1), Divider(1), Divider((uint32_t)p.S), 0, 0};   // no heads: no steps
        const int step = 512 / D, q_blocks = (p.Hq + step - 1) / step, k_blocks = (p.Hkv + step - 1) / step;
        if (q_blocks) plan.by_q = Divider((uint32_t)q_blocks);
        if (k_blocks) plan.by_k = Divider((uint32_t)k_blocks);
        plan.q_units = (int)(tokens * q_blocks);
        plan.k_units = (int)(tokens * k_blocks);
        gsr_rope_bwd_kernel<T, D><<<(unsigned)a.ctas, kThreads, 0, stream>>>(a, plan);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (a.dq_weight || a.dk_weight) {
        cudaLaunchConfig_t cfg{};
        cudaLaunchAttribute early;
        early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        early.val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3(D / 32, 2);
        cfg.blockDim = dim3(1024);
        cfg.stream = stream;
        cfg.attrs = &early;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, gsr_rope_weights_kernel, static_cast<const float*>(a.parts), a.ctas, D, a.dq_weight, a.dk_weight);
    }
    return e;
}

// ---------------------------------------------------------------------------
// Rows of a cache of 4 bits, read back
// ---------------------------------------------------------------------------
// A lane takes 16 values: 8 bytes of codes become 32 bytes.  s x code is exact in fp32, so a value is rounded
// once there and once to T.
template <class T, int D>
__global__ void __launch_bounds__(kThreads) gsr_read4_kernel(const __grid_constant__ Read4Params p, const Divider by_head,
                                                             const Divider by_page, long long rows) {
    constexpr int LANES = D / 16, PER = kThreads / LANES;
    const long long id = (long long)blockIdx.x * PER + threadIdx.x / LANES;      // a token's heads of K, then of V
    const int l = threadIdx.x % LANES;
    if (id >= rows) return;
    const bool is_v = id >= rows / 2;
    const int r = (int)(is_v ? id - rows / 2 : id), n = by_head(r), h = r - n * p.H;
    const int slot = __ldg(p.slots + n);
    if (slot < 0 || slot >= (long long)p.num_pages * p.page) return;
    const long long page = by_page(slot);
    const int row = slot - (int)page * p.page;
    const Cache4& cache = is_v ? p.V4 : p.K4;
    const Strided& to = is_v ? p.V : p.K;
    const uint2 codes = __ldg(reinterpret_cast<const uint2*>(cache.codes.data + page * cache.codes.page +
                                                             (long long)row * cache.codes.row + h * cache.codes.head) + l);
    const float2 sm = Pair<T>::unpack(__ldg(reinterpret_cast<const uint32_t*>(cache.params.data + page * cache.params.page +
                                                                             (long long)row * cache.params.row +
                                                                             h * cache.params.head) + l / 4));
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = fmaf(sm.x, (float)((i < 8 ? codes.x : codes.y) >> (4 * (i & 7)) & 15u), sm.y);
    uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(to.data) + n * to.row + h * to.head) + 2 * l;
    out[0] = pack8<T>(v);
    out[1] = pack8<T>(v + 8);
}

template <class T, int D>
cudaError_t launch_read(const Read4Params& p, cudaStream_t stream) {
    const long long rows = 2ll * p.N * p.H;
    constexpr int PER = kThreads / (D / 16);
    gsr_read4_kernel<T, D><<<(unsigned)((rows + PER - 1) / PER), kThreads, 0, stream>>>(p, Divider((uint32_t)p.H),
                                                                                        Divider((uint32_t)p.page), rows);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_fwd(const RopeParams& p, bool bf16, int sms, cudaStream_t stream) {
    RopeAppendParams a{};
    a.f = p;
    return launch_rope_type<kSinkRows>(a, bf16, sms, stream);
}

cudaError_t launch_rope_append(const RopeAppendParams& p, bool bf16, bool four_bits, int sms, cudaStream_t stream) {
    return four_bits ? launch_rope_type<kSinkCache4>(p, bf16, sms, stream) : launch_rope_type<kSinkCache16>(p, bf16, sms, stream);
}

int rope_bwd_ctas(long long batch, long long heads_q, long long heads_kv, long long seq, int D, int sms) {
    const int rows = 512 / D;
    return rope_ctas(batch * seq * (((heads_q > heads_kv ? heads_q : heads_kv) + rows - 1) / rows), kBwdCtasAnSm * sms);
}

cudaError_t launch_rope_bwd(const RopeBwdParams& p, bool bf16, cudaStream_t stream) {
    if (p.f.D == 64) return bf16 ? launch_bwd<__nv_bfloat16, 64>(p, stream) : launch_bwd<__half, 64>(p, stream);
    return bf16 ? launch_bwd<__nv_bfloat16, 128>(p, stream) : launch_bwd<__half, 128>(p, stream);
}

cudaError_t launch_read4(const Read4Params& p, bool bf16, cudaStream_t stream) {
    if (p.D == 64) return bf16 ? launch_read<__nv_bfloat16, 64>(p, stream) : launch_read<__half, 64>(p, stream);
    return bf16 ? launch_read<__nv_bfloat16, 128>(p, stream) : launch_read<__half, 128>(p, stream);
}

}  // namespace gsr
