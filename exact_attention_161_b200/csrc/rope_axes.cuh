// rope_axes.cuh -- rotary positions with several axes (time, height, width, ...) on packed tokens.
//
// Each of the R/2 rotated pairs of a head belongs to one axis; pair i of token t is rotated by
//   angle = pos[axis(i)][t] / pos_scale * theta_i,
// y0 = x0 cos - x1 sin, y1 = x0 sin + x1 cos, for every head of the token alike. The inverse (the
// gradient of the rotation) turns by -angle. With one axis and positions 0, 1, 2, ... this is RoPE
// ("attention-transformers", Q "How does Rotary Position Embedding (RoPE) work?").
//
// Positions are device data of any int32 value, so there is no table: the angle is formed in
// revolutions in fp64 (pos / pos_scale * theta / 2 pi), reduced to a fraction in [-1/2, 1/2] and handed to
// sincospif in fp32. The constant, the quotient and the product are each off by at most 2^-53 of the
// revolutions, the fraction in fp32 by 2^-26: 1.2e-7 revolutions together at |pos| = 2^31, pos_scale = 1 and
// theta = 1; at smaller theta the power adds its own rounding to fewer revolutions, and a pos_scale below 1
// makes them and the error so many times larger. The products and the sum are fp32; one rounding to bf16 at the store.
//
// Bound: HBM (each element is read and written once). A warp rotates one token's heads (or a share of
// them, where there are few tokens): each lane computes the angles of one or two pairs, once per token and
// not once per head, and passes them on through shared memory; then it keeps the angles of its own 8 pairs
// in registers and walks the heads, five 32-byte pieces in flight. Nothing but the warp is synchronised: a
// version with 256-thread blocks sharing the angles of three tokens waited at its barriers: 32,768 tokens
// of 40 heads of 128 took 154 us against 108 us here (6.2 TB/s). Two pieces in flight: 113 us, ten: 117 us.
#pragma once
#include "common.cuh"
#include "ptx.cuh"

namespace attn {

constexpr int kRopeAxesMax = 8;

struct RopeAxesParams {
    const __nv_bfloat16* src[2];  // [T, heads, D]: q, k
    __nv_bfloat16* dst[2];
    long long src_stride[2], dst_stride[2];  // elements from one token to the next
    const int32_t* pos;           // [axes, T]
    int heads[2];
    int T, half;                  // half: pairs (i, i + R/2) instead of (2i, 2i + 1)
    int share, per_share;         // a token's heads are cut into `share` items of per_share heads
    int pairs;                    // R/2
    float sign;                   // -1 for the inverse
    uint8_t axis[64];             // axis of pair i
    double rev[64];               // theta_i / (2 pi pos_scale): revolutions per position
};

template <int D>
__global__ void __launch_bounds__(128) rope_axes_kernel(const __grid_constant__ RopeAxesParams p) {
    constexpr int PIECES = D / 16;        // of a head: 8 pairs each, or 16 elements that are not rotated
    constexpr int STEP = 32 / PIECES;     // heads a warp takes at a time
    constexpr int U = 5;                  // pieces in flight per lane
    __shared__ __align__(16) float2 s_cs[4][64];
    const int lane = threadIdx.x & 31;
    float2* cs = s_cs[threadIdx.x >> 5];
    const int H = p.heads[0] + p.heads[1], R2 = p.pairs;
    const int c = lane % PIECES;
    const bool rotated = 8 * c < R2;
    // the two halves of this lane's piece: the 8 first and 8 second members of 8 pairs (half-split), 8
    // neighbouring pairs, or 16 elements behind the rotated ones
    const int off1 = p.half && rotated ? 8 * c : 16 * c, off2 = p.half && rotated ? 8 * c + R2 : 16 * c + 8;
    const int pr0 = min(lane, R2 - 1), pr1 = min(lane + 32, R2 - 1);
    const double rev0 = p.rev[pr0], rev1 = p.rev[pr1];
    const int32_t* pos0 = p.pos + static_cast<size_t>(p.axis[pr0]) * p.T;
    const int32_t* pos1 = p.pos + static_cast<size_t>(p.axis[pr1]) * p.T;
    auto angle = [&](int pos, double rev) {
        const double x = static_cast<double>(pos) * rev;
        float sn, co;
        sincospif(2.f * static_cast<float>(x - rint(x)), &sn, &co);
        return make_float2(co, p.sign * sn);
    };
    const long long items = static_cast<long long>(p.T) * p.share;  // (token, share of its heads)
    const long long warps = static_cast<long long>(gridDim.x) * 4;
    for (long long w = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5); w < items; w += warps) {
        const int t = static_cast<int>(w / p.share), part = static_cast<int>(w - static_cast<long long>(t) * p.share);
        const int x0 = pos0[t], x1 = pos1[t];
        const int h_end = min(H, (part + 1) * p.per_share);
        bool ready = false;
        for (int h0 = part * p.per_share + lane / PIECES; h0 - lane / PIECES < h_end; h0 += STEP * U) {
            uint4 a[U], b[U];
            auto row = [&](const auto& base, const long long (&stride)[2], int h) {
                const int z = h >= p.heads[0];
                return base[z] + t * stride[z] + (z ? h - p.heads[0] : h) * D;
            };
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int h = h0 + j * STEP;
                if (h >= h_end) continue;
                const __nv_bfloat16* s = row(p.src, p.src_stride, h);
                a[j] = *reinterpret_cast<const uint4*>(s + off1);
                b[j] = *reinterpret_cast<const uint4*>(s + off2);
            }
            if (!ready) {
                cs[pr0] = angle(x0, rev0);
                if (R2 > 32) cs[pr1] = angle(x1, rev1);
                __syncwarp();
                ready = true;
            }
            float4 k[4];  // this lane's 8 pairs, two each
            if (rotated) {
#pragma unroll
                for (int e = 0; e < 4; ++e) k[e] = reinterpret_cast<const float4*>(cs + 8 * c)[e];
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int h = h0 + j * STEP;
                if (h >= h_end) continue;
                uint4 y0 = a[j], y1 = b[j];
                if (rotated) {
                    const uint32_t u[4] = {a[j].x, a[j].y, a[j].z, a[j].w}, v[4] = {b[j].x, b[j].y, b[j].z, b[j].w};
                    uint32_t r[8];
                    if (p.half) {
                        // u: members x0 of pairs 0..7, v: members x1
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x0 = ptx::bf16lo_to_f32(u[e]), x2 = ptx::bf16hi_to_f32(u[e]);
                            const float x1 = ptx::bf16lo_to_f32(v[e]), x3 = ptx::bf16hi_to_f32(v[e]);
                            r[e] = ptx::pack_bf16x2(x0 * k[e].x - x1 * k[e].y, x2 * k[e].z - x3 * k[e].w);
                            r[4 + e] = ptx::pack_bf16x2(x0 * k[e].y + x1 * k[e].x, x2 * k[e].w + x3 * k[e].z);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t p0 = e < 2 ? u[2 * e] : v[2 * e - 4], p1 = e < 2 ? u[2 * e + 1] : v[2 * e - 3];
                            const float x0 = ptx::bf16lo_to_f32(p0), x1 = ptx::bf16hi_to_f32(p0);
                            const float x2 = ptx::bf16lo_to_f32(p1), x3 = ptx::bf16hi_to_f32(p1);
                            r[2 * e] = ptx::pack_bf16x2(x0 * k[e].x - x1 * k[e].y, x0 * k[e].y + x1 * k[e].x);
                            r[2 * e + 1] = ptx::pack_bf16x2(x2 * k[e].z - x3 * k[e].w, x2 * k[e].w + x3 * k[e].z);
                        }
                    }
                    y0 = make_uint4(r[0], r[1], r[2], r[3]);
                    y1 = make_uint4(r[4], r[5], r[6], r[7]);
                }
                __nv_bfloat16* out = row(p.dst, p.dst_stride, h);
                *reinterpret_cast<uint4*>(out + off1) = y0;
                *reinterpret_cast<uint4*>(out + off2) = y1;
            }
        }
        __syncwarp();  // the next token's angles overwrite cs
    }
}

}  // namespace attn
