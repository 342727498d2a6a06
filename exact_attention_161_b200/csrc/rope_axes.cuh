// rope_axes.cuh -- rotary positions with several axes (time, height, width, ...) on packed tokens.
//
// Each of the R/2 rotated pairs of a head belongs to one axis; pair i of token t is rotated by
//   angle = pos[axis(i)][t] / pos_scale * theta_i,
// y0 = x0 cos - x1 sin, y1 = x0 sin + x1 cos, for every head of the token alike. The inverse (the
// gradient of the rotation) turns by -angle. With one axis and positions 0, 1, 2, ... this is RoPE
// ("attention-transformers", Q "How does Rotary Position Embedding (RoPE) work?").
//
// Positions are device data of any int32 value, so there is no table: the angle is formed in
// revolutions in fp64 (pos * theta / 2 pi: positions far out lose nothing; at |pos| = 2^31 the
// fraction is right to 4e-8 revolutions), reduced to a fraction in [-1/2, 1/2] and handed to
// sincospif in fp32. The products and the sum are fp32; one rounding to bf16 at the store.
//
// Bound: HBM (each element is read and written once). One CTA rotates `group` tokens at a time: a
// thread computes the angle of one (token, pair) into shared memory, so that the fp64 work and the
// sincos are paid once per token, not once per head; then the CTA's threads walk the tokens' (head,
// 16-element piece) items, loading several before the angles are needed.
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
    int T, group, half;           // half: pairs (i, i + R/2) instead of (2i, 2i + 1)
    int pairs;                    // R/2
    float sign;                   // -1 for the inverse
    uint8_t axis[64];             // axis of pair i
    double rev[64];               // theta_i / (2 pi pos_scale): revolutions per position
};

template <int D>
__global__ void __launch_bounds__(256) rope_axes_kernel(const __grid_constant__ RopeAxesParams p) {
    constexpr int PIECES = D / 16;  // of a head: 8 pairs each, or 16 elements that are not rotated
    constexpr int U = 4;            // items in flight per thread
    constexpr int kMaxGroup = 16;
    __shared__ float2 s_cs[kMaxGroup * 64];
    const int H = p.heads[0] + p.heads[1];
    const int R2 = p.pairs;
    for (int t0 = blockIdx.x * p.group; t0 < p.T; t0 += gridDim.x * p.group) {
        const int n = min(p.group, p.T - t0);
        const int items = n * H * PIECES;
        for (int base = 0; base < items || base == 0; base += 256 * U) {
            uint4 a[U], b[U];
            int tok[U], piece[U];
            __nv_bfloat16* out[U];
            // 16 elements of one head: the 8 first and 8 second members of 8 pairs (half-split), 8
            // neighbouring pairs, or 16 elements behind the rotated ones
            auto offset1 = [&](int c) { return p.half && 8 * c < R2 ? 8 * c : 16 * c; };
            auto offset2 = [&](int c) { return p.half && 8 * c < R2 ? 8 * c + R2 : 16 * c + 8; };
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int idx = base + j * 256 + threadIdx.x;
                tok[j] = -1;
                if (idx >= items) continue;
                const int c = idx % PIECES, th = idx / PIECES;
                const int t = th / H, h = th - t * H;
                const int z = h >= p.heads[0];
                const int hz = z ? h - p.heads[0] : h;
                const __nv_bfloat16* s = (z ? p.src[1] + (t0 + t) * p.src_stride[1] : p.src[0] + (t0 + t) * p.src_stride[0]) + hz * D;
                out[j] = (z ? p.dst[1] + (t0 + t) * p.dst_stride[1] : p.dst[0] + (t0 + t) * p.dst_stride[0]) + hz * D;
                tok[j] = t;
                piece[j] = c;
                a[j] = *reinterpret_cast<const uint4*>(s + offset1(c));
                b[j] = *reinterpret_cast<const uint4*>(s + offset2(c));
            }
            if (base == 0) {
                for (int i = threadIdx.x; i < n * R2; i += 256) {
                    const int t = i / R2, pr = i - t * R2;
                    const double x = static_cast<double>(p.pos[static_cast<size_t>(p.axis[pr]) * p.T + t0 + t]) * p.rev[pr];
                    float sn, cs;
                    sincospif(2.f * static_cast<float>(x - rint(x)), &sn, &cs);
                    s_cs[t * 64 + pr] = make_float2(cs, p.sign * sn);
                }
                __syncthreads();
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (tok[j] < 0) continue;
                const int c = piece[j];
                uint4 y0 = a[j], y1 = b[j];
                if (8 * c < R2) {
                    const float4* cs = reinterpret_cast<const float4*>(s_cs + tok[j] * 64 + 8 * c);  // two pairs each
                    const uint32_t u[4] = {a[j].x, a[j].y, a[j].z, a[j].w}, v[4] = {b[j].x, b[j].y, b[j].z, b[j].w};
                    uint32_t w[8];
                    if (p.half) {
                        // u: members x0 of pairs 0..7, v: members x1
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 k = cs[e];
                            const float x0 = ptx::bf16lo_to_f32(u[e]), x2 = ptx::bf16hi_to_f32(u[e]);
                            const float x1 = ptx::bf16lo_to_f32(v[e]), x3 = ptx::bf16hi_to_f32(v[e]);
                            w[e] = ptx::pack_bf16x2(x0 * k.x - x1 * k.y, x2 * k.z - x3 * k.w);
                            w[4 + e] = ptx::pack_bf16x2(x0 * k.y + x1 * k.x, x2 * k.w + x3 * k.z);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 k = cs[e];
                            const uint32_t p0 = e < 2 ? u[2 * e] : v[2 * e - 4], p1 = e < 2 ? u[2 * e + 1] : v[2 * e - 3];
                            const float x0 = ptx::bf16lo_to_f32(p0), x1 = ptx::bf16hi_to_f32(p0);
                            const float x2 = ptx::bf16lo_to_f32(p1), x3 = ptx::bf16hi_to_f32(p1);
                            w[2 * e] = ptx::pack_bf16x2(x0 * k.x - x1 * k.y, x0 * k.y + x1 * k.x);
                            w[2 * e + 1] = ptx::pack_bf16x2(x2 * k.z - x3 * k.w, x2 * k.w + x3 * k.z);
                        }
                    }
                    y0 = make_uint4(w[0], w[1], w[2], w[3]);
                    y1 = make_uint4(w[4], w[5], w[6], w[7]);
                }
                *reinterpret_cast<uint4*>(out[j] + offset1(c)) = y0;
                *reinterpret_cast<uint4*>(out[j] + offset2(c)) = y1;
            }
        }
        __syncthreads();  // the next tokens' angles overwrite s_cs
    }
}

}  // namespace attn
