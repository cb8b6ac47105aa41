// ckpt_qk.cu -- RMS norm of every query and key head with the position rotation
// in the same pass, keeping the heads as an 8-bit checkpoint, and its backward
// pass from that checkpoint (COAT review page, section 3: FP8 activations,
// 1 x G groups for non-linear layers).
//
//   forward   per head x of D: r = 1 / sqrt(mean x^2 + eps), y = x r w, then the
//             first rot entries of y are turned in pairs (a, b) by the angle of
//             the token's position: (a c - b s, b c + a s).  Pairs are
//             (i, i + rot/2), or (2i, 2i + 1) when interleaved.
//   backward  dn = the gradient turned back, g = dn w, xh = S E4M3(q) r:
//             dx = r (g - xh mean(g xh));  dw = sum over tokens and heads of dn xh
//
// Everything between input and output is float32, rounded once to bf16.
//
// A head lies in D / 16 lanes (the next power of two of them; the others idle)
// that hold two chunks of eight entries each, so that its sums are a few
// shuffles.  The chunks are chosen so that both entries of a pair are in one
// thread: lane l < rot / 16 has entries 8 l and rot / 2 + 8 l onwards when the
// pairs are split, and every other lane 16 l onwards.  Eight cosines and
// sines per lane then serve all heads of a token, and stay in registers as
// factors of an entry and of its partner.  A block works for one of the two
// sides, so that a lane has one set of weights and, backward, of sums for dw.
// Forward a warp takes one token's heads of its side, or a share of them;
// backward, where blocks have to stay for their sums, the passes over the
// tokens' heads go to the warps in equal ranges.
//
// Both directions are bound by memory in the long run (time per further token:
// the copy rate forward, 85 to 93 % of it backward) and are sensitive to two
// things.  Registers: three blocks of 256 threads with 80 registers, some of
// them in local memory, took 61.6 us forward at 8192 tokens x 64 heads x 128
// where nine of 64 threads take 54.8.  And the balance of the warps' work: equal
// ranges of passes instead of tokens brought 4101 tokens x 50 heads x 128
// backward from 35.9 to 31.1 us (30.5 now), of which 7 to 8 do not grow with the tokens (two kernels, first passes).
#include <cstdint>

#include "ckpt_device.cuh"
#include "ckpt_kernels.h"

namespace coat {

namespace {

using namespace ckpt;

constexpr int kFwdBlock = 64;          // threads of a block, forward
constexpr int kFwdWarps = kFwdBlock / 32;
constexpr int kFwdPerSm = 9;           // blocks that the registers allow
constexpr int kFwdPasses = 8;          // passes over heads that a warp makes for a token at most
constexpr int kBlock = 128;            // backward
constexpr int kWarps = kBlock / 32;
constexpr int kPerSm = 3;

// How a group's maximum is found.
enum GroupMode {
    kAdjacent,   // a lane's chunks lie together: G = 16 is a lane, G / 16 lanes beyond
    kSplit,      // lane l has chunks l and l + D / 16: G / 8 lanes each, or all lanes together (G = D)
    kMixed       // anything else: chunk by chunk
};

// Forward: 2^shift warps share a token's heads of one side, `passes` passes (of the warp's lanes over heads) each.
struct Split {
    int32_t shift, passes;
};
struct Task {
    int64_t blocks_q;    // blocks below: queries; the others: keys
    Split q, k;
    int32_t mode;
};

__device__ __forceinline__ void load8f(const float* p, float* x) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// The first entries of a lane's chunks.
struct Place {
    int a, b;
};
__device__ __forceinline__ Place place_of(int l, int rot, bool interleaved) {
    const bool split = !interleaved && 16 * l < rot;
    return split ? Place{8 * l, rot / 2 + 8 * l} : Place{16 * l, 16 * l + 8};
}

// Cosines and sines of a lane's eight pairs; 1 and 0 behind rot, NaN at a position outside the tables.
__device__ __forceinline__ void load_turn(const QkArgs& a, int64_t m, int l, float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) { c[e] = 1.0f; s[e] = 0.0f; }
    if (16 * l >= a.rot) return;
    const int64_t pos = a.positions[m];
    if (pos >= 0 && pos < a.max_pos) {
        load8f(a.cos + pos * (a.rot / 2) + 8 * l, c);
        load8f(a.sin + pos * (a.rot / 2) + 8 * l, s);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = s[e] = __uint_as_float(0x7FC00000u);
    }
}

// A lane's sixteen entries as pairs, chunk after chunk.  The partner of pair e's entries: the pair of the other chunk
// (split), or the pair itself, swapped (interleaved).
template <bool kInter>
__device__ __forceinline__ uint64_t partner(const uint64_t (&x)[8], int e) {
    if (!kInter) return x[e ^ 4];
    float lo, hi;
    upk(x[e], lo, hi);
    return pk(hi, lo);
}
// The turn by the angles as out = x own + partner(x) other, the factors in the entries' order.  w: the entries' weights,
// folded in (ones backward); kBack: the angles' signs turned.  (Lanes behind rot hold entries that do not pair: their
// angle is 0.)
template <bool kInter, bool kBack>
__device__ __forceinline__ void turn_factors(const float (&c)[8], const float (&s)[8], const float (&w)[16], uint64_t (&own)[8],
                                             uint64_t (&other)[8]) {
    float o[16], p[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int ia = kInter ? 2 * i : i, ib = kInter ? 2 * i + 1 : i + 8;
        o[ia] = w[ia] * c[i];
        o[ib] = w[ib] * c[i];
        p[ia] = kBack ? w[ib] * s[i] : -(w[ib] * s[i]);
        p[ib] = kBack ? -(w[ia] * s[i]) : w[ia] * s[i];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        own[e] = pk(o[2 * e], o[2 * e + 1]);
        other[e] = pk(p[2 * e], p[2 * e + 1]);
    }
}
__device__ __forceinline__ void load8f2(const float* p, uint64_t* x) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p), b = reinterpret_cast<const ulonglong2*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}

template <int kLanes>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}

// Group maxima of the two chunks of every lane (bf16 values; idle lanes have zeros).
__device__ __forceinline__ void group_maxima(float& ma, float& mb, int mode, int lanes, int l, int base, const QkArgs& a) {
    if (a.G == 8) return;
    if (mode == kAdjacent) {
        ma = mb = lanes_max(fmaxf(ma, mb), a.G >> 4);
        return;
    }
    if (mode == kSplit && a.G == a.D) {
        ma = mb = lanes_max(fmaxf(ma, mb), lanes);
        return;
    }
    // both maxima in one word: a bf16 value is the upper half of its float
    uint32_t v = __byte_perm(__float_as_uint(ma), __float_as_uint(mb), 0x7632);
    if (mode == kSplit) {
        for (int off = a.G >> 4; off > 0; off >>= 1) {
            const uint32_t o = __shfl_xor_sync(kFull, v, off);
            asm("max.u16x2 %0, %0, %1;" : "+r"(v) : "r"(o));
        }
        ma = __uint_as_float(v << 16);
        mb = __uint_as_float(v & 0xFFFF0000u);
        return;
    }
    const int per = a.G >> 3, rl = a.rot >> 4;    // chunks of a group; lanes with split pairs
    const Place p = place_of(l, a.rot, a.interleaved != 0);
    const int ga = (p.a >> 3) & ~(per - 1), gb = (p.b >> 3) & ~(per - 1);
    uint32_t wa = 0u, wb = 0u;
    for (int j = 0; j < 2 * per; ++j) {
        const int c = j < per ? ga + j : gb + j - per;
        const bool second = c < 2 * rl ? c >= rl : (c & 1) != 0;
        const int from = c < 2 * rl ? (second ? c - rl : c) : c >> 1;
        const uint32_t o = __shfl_sync(kFull, v, base + from);
        const uint32_t x = second ? o >> 16 : o & 0xFFFFu;
        if (j < per) wa = wa > x ? wa : x;
        else wb = wb > x ? wb : x;
    }
    ma = __uint_as_float(wa << 16);
    mb = __uint_as_float(wb << 16);
}

__device__ __forceinline__ void store_pair(uint16_t* p, const Place& at, const uint32_t (&w)[8]) {
    *reinterpret_cast<uint4*>(p + at.a) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(p + at.b) = make_uint4(w[4], w[5], w[6], w[7]);
}

// What a lane will need in the next passes, copied into its own place in shared
// memory asynchronously: three passes on their way without registers.
constexpr int kRing = 4;
template <int n>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (n == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but this thread's last n groups have landed, 1 <= n <= 3
__device__ __forceinline__ void cp_async_wait(int n) {
    if (n == 3)
        asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (n == 2)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 1;" ::: "memory");
}
static_assert(kRing == 4, "cp_async_wait");

// The output and 1 / rms of those of a warp's heads, `from` to `to` of token m, whose mean square left float32's range (the
// usual path has written NaN): the sum is formed of kFar times the entries.  The whole warp comes here, behind its last
// pass, and takes everything from memory, so that the passes only note that there is such a head.
__device__ __noinline__ void far_heads(const QkArgs& a, const HeadSide& sd, int64_t m, int from, int to, int lane) {
    __syncwarp();                              // the lanes see each other's 1 / rms
    const int64_t pos = a.positions[m];
    const int half = a.rot / 2;
    for (int h = from; h < to; ++h) {
        const int64_t row = m * sd.H + h;
        if (sd.rstd[row] > 0.0f) continue;
        const uint16_t* x = sd.in + m * sd.ld + (int64_t)h * a.D;
        auto entry = [&](int c) { return __uint_as_float((uint32_t)x[c] << 16) * kFar; };
        float ss = 0.0f;
        for (int c = lane; c < a.D; c += 32) ss = fmaf(entry(c), entry(c), ss);
        const float r = far_rsqrt(fmaf(warp_sum(ss), 1.0f / (float)a.D, a.eps * kFar * kFar));
        for (int c = lane; c < a.D; c += 32) {
            float y = entry(c) * sd.weight[c];
            if (c < a.rot) {
                const bool second = a.interleaved ? (c & 1) != 0 : c >= half;
                const int i = a.interleaved ? c >> 1 : second ? c - half : c;      // the pair, and its other entry
                const int p = a.interleaved ? c ^ 1 : second ? c - half : c + half;
                const bool in = pos >= 0 && pos < a.max_pos;
                const float co = in ? a.cos[pos * half + i] : __uint_as_float(0x7FC00000u);
                const float si = in ? a.sin[pos * half + i] : co;
                const float z = entry(p) * sd.weight[p] * si;
                y = fmaf(y, co, second ? z : -z);
            }
            sd.out[row * a.D + c] = bf16_bits(y * r);
        }
        __syncwarp();
        if (lane == 0) sd.rstd[row] = r * kFar;
    }
}

template <int kLanes, bool kInter>
__global__ void __launch_bounds__(kFwdBlock, kFwdPerSm) qk_fwd_kernel(const __grid_constant__ QkArgs a, const Task tk) {
    constexpr int kHeads = 32 / kLanes;   // heads per warp and pass
    const int lane = threadIdx.x & 31, l = lane & (kLanes - 1), base = lane - l, sub = lane / kLanes;
    const bool is_q = blockIdx.x < tk.blocks_q;
    const HeadSide sd = is_q ? a.q : a.k;
    const Split sp = is_q ? tk.q : tk.k;
    const int64_t t = (int64_t)(blockIdx.x - (is_q ? 0 : tk.blocks_q)) * kFwdWarps + (threadIdx.x >> 5);
    const int64_t m = t >> sp.shift;
    if (m >= a.M) return;
    const int from = ((int)t & ((1 << sp.shift) - 1)) * sp.passes;
    const int to = min(from + sp.passes, (sd.H + kHeads - 1) / kHeads);
    const bool in_head = l * 16 < a.D;
    const Place at = place_of(l, a.rot, kInter);
    const uint16_t* in = sd.in + m * sd.ld;
    const int64_t row = m * sd.H;         // head 0 of this token
    const int gshift = 31 - __clz(a.G), gpr = a.D >> gshift;
    const float inv_d = 1.0f / (float)a.D;
    __shared__ uint4 ring[kRing][2][kFwdBlock];
    wait_for_primary();
    const int h0 = from * kHeads + sub;
    const uint16_t* next = in + (int64_t)h0 * a.D;
    auto fetch = [&](int i) {                            // pass from + i, if there is one
        if (from + i < to && in_head && h0 + i * kHeads < sd.H) {
            cp_async<16>(&ring[i & (kRing - 1)][0][threadIdx.x], next + at.a);
            cp_async<16>(&ring[i & (kRing - 1)][1][threadIdx.x], next + at.b);
        }
        cp_async_commit();
        next += kHeads * a.D;
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) fetch(i);
    uint64_t own[8], other[8];
    {
        float c[8], s[8], w[16] = {};
        load_turn(a, m, l, c, s);
        if (in_head) {
            load8f(sd.weight + at.a, w);
            load8f(sd.weight + at.b, w + 8);
        }
        turn_factors<kInter, false>(c, s, w, own, other);
    }
    const bool one_scale = tk.mode == kAdjacent ? a.G > 8 : tk.mode == kSplit && a.G == a.D;
    const bool first_a = (at.a & (a.G - 1)) == 0, first_b = (at.b & (a.G - 1)) == 0;
    int64_t hd = (row + h0) * a.D;                       // the head's place in the outputs
    float* sc = sd.scale + (row + h0) * gpr;
    float* rs = sd.rstd + row + h0;
    bool far = false;
    for (int i = 0, h = h0; from + i < to; ++i, h += kHeads) {
        const bool ok = in_head && h < sd.H;
        fetch(i + kRing - 1);
        cp_async_wait(kRing - 1);
        uint64_t x2[8] = {}, ss2 = 0ull;
        if (ok) {
            const uint4* src = &ring[i & (kRing - 1)][0][threadIdx.x];
            const uint4 lo = src[0], hi = src[kFwdBlock];
            const uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            unpack2(u, x2);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ss2 = fma2(x2[e], x2[e], ss2);
        const float ss = head_sum<kLanes>(sum2(ss2));
        const float v = fmaf(ss, inv_d, a.eps), r = rsqrt_newton(v);
        far |= !(v < INFINITY);
        float ma = max_of<0, 4>(x2), mb = max_of<4, 4>(x2);
        group_maxima(ma, mb, tk.mode, kLanes, l, base, a);
        const Scale sa = scale_of_bf16_max(ma);
        Scale sb = sa;
        if (!one_scale) sb = scale_of_bf16_max(mb);
        uint32_t q[4], o[8];
        encode16(x2, sa, sb, q);
        const uint64_t r2 = pk(r, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float lo, hi;
            upk(mul2(fma2(partner<kInter>(x2, e), other[e], mul2(x2[e], own[e])), r2), lo, hi);
            o[e] = bf16x2(lo, hi);
        }
        if (ok) {
            store_pair(sd.out + hd, at, o);
            *reinterpret_cast<uint2*>(sd.codes + hd + at.a) = make_uint2(q[0], q[1]);
            *reinterpret_cast<uint2*>(sd.codes + hd + at.b) = make_uint2(q[2], q[3]);
            if (first_a) sc[at.a >> gshift] = sa.S;
            if (first_b) sc[at.b >> gshift] = sb.S;
            if (l == 0) *rs = r;
        }
        hd += kHeads * a.D;
        sc += kHeads * gpr;
        rs += kHeads;
    }
    if (__any_sync(kFull, far)) far_heads(a, is_q ? a.q : a.k, m, from * kHeads, min(to * kHeads, sd.H), lane);
}

// A lane's ring, and the angles of its token and of the next one.
struct BwdShared {
    uint4 dy[kRing][2][kBlock];
    uint2 q[kRing][2][kBlock];
    float s[kRing][3][kBlock];     // the chunks' scales, and 1 / rms
    float4 angle[2][4][kBlock];    // eight cosines, eight sines
};

// The passes of a side's tokens, in order, go to its warps in equal ranges.
template <int kLanes, bool kInter>
__global__ void __launch_bounds__(kBlock, kPerSm) qk_bwd_kernel(const QkArgs a, const Task tk) {
    constexpr int kHeads = 32 / kLanes;
    __shared__ BwdShared sh;
    const int lane = threadIdx.x & 31, l = lane & (kLanes - 1), sub = lane / kLanes, warp = threadIdx.x >> 5;
    const bool is_q = blockIdx.x < tk.blocks_q;
    const HeadSide sd = is_q ? a.q : a.k;
    const int64_t blocks = is_q ? tk.blocks_q : gridDim.x - tk.blocks_q;
    const int64_t me = (int64_t)(blockIdx.x - (is_q ? 0 : tk.blocks_q)) * kWarps + warp;
    const int passes = (sd.H + kHeads - 1) / kHeads;
    const bool in_head = l * 16 < a.D, turned = l * 16 < a.rot;
    const Place at = place_of(l, a.rot, kInter);
    const int gshift = 31 - __clz(a.G), to_b = at.b - at.a;
    const float inv_d = 1.0f / (float)a.D;
    uint64_t w[8] = {}, dw2[8] = {};
    wait_for_primary();
    if (in_head) {
        load8f2(sd.weight + at.a, w);
        load8f2(sd.weight + at.b, w + 4);
    }
    const int64_t all = a.M * passes, warps = blocks * kWarps;
    const int64_t from = all / warps * me + min(me, all % warps);
    int left = (int)(all / warps + (me < all % warps ? 1 : 0));          // passes to do, and to fetch
    int fetches = left;
    int64_t m = from / passes;
    int p = (int)(from - m * passes), fp = p;
    const int last = (passes - 1) * kHeads;
    int64_t frow = m * sd.H + p * kHeads + sub;                          // the row (token, head) that is fetched next
    uint16_t* out = sd.out + m * sd.ld + (int64_t)(p * kHeads + sub) * a.D + at.a;
    // A token's angles come with its first pass; fetched are at most as many passes ahead as a token has, so that there
    // are never more than two tokens' angles.
    const int ahead = min(kRing - 1, passes);
    auto position = [&](int64_t t) { return turned && t < a.M ? (int64_t)a.positions[t] : (int64_t)-1; };
    int64_t fm = m, pos = left > 0 ? position(m) : -1;
    uint32_t known = 0u, place = 0u, fplace = 0u;     // known: a bit per place: the position is in the tables
    bool fresh = true;
    auto fetch = [&](int u) {
        if (fetches > 0) {
            if (fresh) {
                const bool in = pos >= 0 && pos < a.max_pos;
                if (in) {
                    const int64_t t = pos * (a.rot / 2) + 8 * l;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        cp_async<16>(&sh.angle[fplace][i][threadIdx.x], a.cos + t + 4 * i);
                        cp_async<16>(&sh.angle[fplace][i + 2][threadIdx.x], a.sin + t + 4 * i);
                    }
                }
                known = (known & ~(1u << fplace)) | ((in ? 1u : 0u) << fplace);
                pos = position(++fm);
                fplace ^= 1u;
                fresh = false;
            }
            if (in_head && fp * kHeads + sub < sd.H) {
                const int64_t off = frow * a.D + at.a;
                cp_async<16>(&sh.dy[u][0][threadIdx.x], sd.in + off);
                cp_async<16>(&sh.dy[u][1][threadIdx.x], sd.in + off + to_b);
                cp_async<8>(&sh.q[u][0][threadIdx.x], sd.codes + off);
                cp_async<8>(&sh.q[u][1][threadIdx.x], sd.codes + off + to_b);
                cp_async<4>(&sh.s[u][0][threadIdx.x], sd.scale + (off >> gshift));
                cp_async<4>(&sh.s[u][1][threadIdx.x], sd.scale + ((off + to_b) >> gshift));
                cp_async<4>(&sh.s[u][2][threadIdx.x], sd.rstd + frow);
            }
            --fetches;
            frow += kHeads;
            if (++fp == passes) {
                fp = 0;
                frow += sd.H - last - kHeads;
                fresh = true;
            }
        }
        cp_async_commit();
    };
    for (int i = 0; i < ahead; ++i) fetch(i);
    uint64_t own[8], other[8];
    bool begins = true;
    for (int u = 0; left > 0; --left, u = (u + 1) & (kRing - 1)) {
        fetch((u + ahead) & (kRing - 1));
        cp_async_wait(ahead);
        if (begins) {
            begins = false;
            float c[8], s[8], one[16];
#pragma unroll
            for (int e = 0; e < 8; ++e) { c[e] = 1.0f; s[e] = 0.0f; }
            if (turned) {
                if ((known >> place) & 1u) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float4 cv = sh.angle[place][i][threadIdx.x], sv = sh.angle[place][i + 2][threadIdx.x];
                        c[4 * i] = cv.x; c[4 * i + 1] = cv.y; c[4 * i + 2] = cv.z; c[4 * i + 3] = cv.w;
                        s[4 * i] = sv.x; s[4 * i + 1] = sv.y; s[4 * i + 2] = sv.z; s[4 * i + 3] = sv.w;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) c[e] = s[e] = __uint_as_float(0x7FC00000u);
                }
            }
            place ^= 1u;
#pragma unroll
            for (int e = 0; e < 16; ++e) one[e] = 1.0f;
            turn_factors<kInter, true>(c, s, one, own, other);
        }
        const bool ok = in_head && p * kHeads + sub < sd.H;
        float xf[16], r = 0.0f, sa = 0.0f, sb = 0.0f;
        uint64_t d2[8] = {}, g2[8], xh[8], k2 = 0ull;
        uint32_t nq[4] = {};
        if (ok) {
            const uint4 lo = sh.dy[u][0][threadIdx.x], hi = sh.dy[u][1][threadIdx.x];
            const uint32_t v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            unpack2(v, d2);
            const uint2 qa = sh.q[u][0][threadIdx.x], qb = sh.q[u][1][threadIdx.x];
            nq[0] = qa.x; nq[1] = qa.y; nq[2] = qb.x; nq[3] = qb.y;
            r = sh.s[u][2][threadIdx.x];
            sa = sh.s[u][0][threadIdx.x] * r;
            sb = sh.s[u][1][threadIdx.x] * r;
        }
        decode(nq, xf);
        const uint64_t sa2 = pk(sa, sa), sb2 = pk(sb, sb);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            xh[e] = mul2(pk(xf[2 * e], xf[2 * e + 1]), e < 4 ? sa2 : sb2);
            g2[e] = fma2(partner<kInter>(d2, e), other[e], mul2(d2[e], own[e]));
            if (ok) dw2[e] = fma2(g2[e], xh[e], dw2[e]);
            g2[e] = mul2(g2[e], w[e]);
            k2 = fma2(g2[e], xh[e], k2);
        }
        const float k = -head_sum<kLanes>(sum2(k2)) * inv_d;
        const uint64_t kk = pk(k, k), rr = pk(r, r);
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float lo, hi;
            upk(mul2(fma2(xh[e], kk, g2[e]), rr), lo, hi);
            o[e] = bf16x2(lo, hi);
        }
        if (ok) {
            *reinterpret_cast<uint4*>(out) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(out + to_b) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        out += kHeads * a.D;
        if (++p == passes) {
            p = 0;
            out += sd.ld - (int64_t)(last + kHeads) * a.D;
            begins = true;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    dependents_may_start();
    // the block's sums: the warp's heads by shuffles, then its warps in order, where the rings were (beside them they would
    // take a block of D = 256 past the 48 KB of static shared memory)
    float(*part_sum)[16 * kLanes] = reinterpret_cast<float(*)[16 * kLanes]>(&sh);
    static_assert(sizeof(float) * kWarps * 16 * kLanes <= sizeof(sh) && sizeof(sh) <= 48 << 10, "shared memory");
    float dw[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) upk(dw2[e], dw[2 * e], dw[2 * e + 1]);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
        for (int off = 16; off >= kLanes; off >>= 1) dw[e] += __shfl_xor_sync(kFull, dw[e], off);
    }
    __syncthreads();                           // every warp is done with its ring
    if (sub == 0 && in_head) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            part_sum[warp][at.a + e] = dw[e];
            part_sum[warp][at.b + e] = dw[8 + e];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.D; i += kBlock) {
        float v = 0.0f;
#pragma unroll
        for (int p2 = 0; p2 < kWarps; ++p2) v += part_sum[p2][i];
        a.partial[(int64_t)blockIdx.x * a.D + i] = v;
    }
}

template <int kLanes, bool kInter>
cudaError_t launch(const QkArgs& a, const Task& tk, bool back, int64_t blocks, cudaStream_t s) {
    if (back)
        return launch_next(qk_bwd_kernel<kLanes, kInter>, (unsigned)blocks, kBlock, 0, s, a, tk);
    return launch_next(qk_fwd_kernel<kLanes, kInter>, (unsigned)blocks, kFwdBlock, 0, s, a, tk);
}
template <int kLanes>
cudaError_t launch(const QkArgs& a, const Task& tk, bool back, int64_t blocks, cudaStream_t s) {
    return a.interleaved ? launch<kLanes, true>(a, tk, back, blocks, s) : launch<kLanes, false>(a, tk, back, blocks, s);
}
int lanes_of(int D) {
    int n = 1;
    while (16 * n < D) n *= 2;
    return n;
}
cudaError_t launch_any(const QkArgs& a, const Task& tk, bool back, int64_t blocks, cudaStream_t s) {
    switch (lanes_of(a.D)) {
        case 1: return launch<1>(a, tk, back, blocks, s);
        case 2: return launch<2>(a, tk, back, blocks, s);
        case 4: return launch<4>(a, tk, back, blocks, s);
        case 8: return launch<8>(a, tk, back, blocks, s);
        default: return launch<16>(a, tk, back, blocks, s);
    }
}

int mode_of(const QkArgs& a) {
    if (a.interleaved) return kAdjacent;
    if (a.rot == a.D && (a.G == a.D || a.D / 2 % a.G == 0)) return kSplit;
    return kMixed;
}

// At most kFwdPasses passes each, so that the angles serve several heads; more warps per token while there are too few
// tokens to give every SM sixteen warps.
Split split_of(int64_t M, int H, int lanes, int sms) {
    const int passes = (H * lanes + 31) / 32;
    Split sp{0, passes};
    while (sp.passes > 1 && (sp.passes > kFwdPasses || (M << sp.shift) < (int64_t)sms * 16)) {
        ++sp.shift;
        sp.passes = (passes + (1 << sp.shift) - 1) >> sp.shift;
    }
    return sp;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

int64_t qk_bwd_partials(int sms) { return (int64_t)sms * kPerSm + 2; }

cudaError_t launch_qk_fwd(const QkArgs& a, cudaStream_t s) {
    const int sms = device_sms(), lanes = lanes_of(a.D);
    Task tk{0, split_of(a.M, a.q.H, lanes, sms), split_of(a.M, a.k.H, lanes, sms), mode_of(a)};
    tk.blocks_q = a.q.H > 0 ? ceil_div(a.M << tk.q.shift, kFwdWarps) : 0;
    const int64_t blocks_k = a.k.H > 0 ? ceil_div(a.M << tk.k.shift, kFwdWarps) : 0;
    if (tk.blocks_q + blocks_k >= (1LL << 31)) return cudaErrorInvalidValue;
    return launch_any(a, tk, false, tk.blocks_q + blocks_k, s);
}

cudaError_t launch_qk_bwd(const QkArgs& a, cudaStream_t s) {
    const int sms = device_sms(), lanes = lanes_of(a.D);
    Task tk{0, Split{0, 0}, Split{0, 0}, mode_of(a)};
    // as many blocks as run at once, shared between the sides as their passes are, one at least where there are heads
    const int64_t room = (int64_t)sms * kPerSm, pq = (a.q.H * lanes + 31) / 32, pk = (a.k.H * lanes + 31) / 32;
    int64_t bq = room * pq / (pq + pk), bk = room - bq;
    const int64_t need_q = ceil_div(a.M * pq, kWarps), need_k = ceil_div(a.M * pk, kWarps);
    bq = a.q.H > 0 ? (bq < 1 ? 1 : bq > need_q ? need_q : bq) : 0;
    bk = a.k.H > 0 ? (bk < 1 ? 1 : bk > need_k ? need_k : bk) : 0;
    tk.blocks_q = bq;
    cudaError_t e = launch_any(a, tk, true, bq + bk, s);
    if (e != cudaSuccess) return e;
    return launch_column_sums(ColumnSum{a.partial, bq, a.q.dweight}, ColumnSum{a.partial + bq * a.D, bk, a.k.dweight}, a.D, s);
}

}  // namespace coat
