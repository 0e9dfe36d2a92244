// Dense product of block-scaled E4M3 codes with its epilogue:
//   z[m, n] = sum_kb x_s[m, kb] w_s[n / 128, kb] sum_{k in kb} x_q[m, k] w[n, k] + bias[n]
//   out[m, n] = bf16(act(z)[m, n] + residual[m, n])
// over K-blocks kb of 128.  With SwiGLU act(z)[m, j] = silu(z[m, j]) z[m, I + j].
//
// One 64 x 64 tile per workgroup (32 gate and 32 up columns with SwiGLU).
#include "common.h"
#include "linear.h"

namespace moe {

namespace {

__device__ __forceinline__ float silu(float z) {
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896340736f));
}
// tanh form: 0.5 z (1 + tanh(u)) = z / (1 + e^-2u), u = sqrt(2 / pi) (z + 0.044715 z^3)
__device__ __forceinline__ float gelu(float z) {
    const float u2 = 1.5957691216057308f * (z + 0.044715f * z * z * z);
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u2 * -1.44269504088896340736f));
}

__global__ void __launch_bounds__(256)
linear_kernel(LinearArgs g) {
    __shared__ uint8_t p[64][144], q[64][144];
    const int tid = threadIdx.x, l = tid & 63, w = tid >> 6, wp = w & 1, wq = w >> 1;
    const bool sw = g.act == kActSwiglu;
    const int64_t m0 = (int64_t)blockIdx.x * 64;
    const int c0 = blockIdx.y * (sw ? 32 : 64);
    const int nkb = g.K / 128;
    // tile column c (0..63) -> weight row: SwiGLU tiles pair gate and up rows
    // in the two 16-column halves of a wave
    auto wrow = [&](int c) -> int {
        if (!sw) return c0 + c < g.N ? c0 + c : -1;
        const int j = c0 + (c >> 5) * 16 + (c & 15);
        return j < g.n_out ? j + ((c >> 4) & 1) * g.n_out : -1;
    };
    v4f acc[2][2] = {};
    for (int kb = 0; kb < nkb; ++kb) {
        __syncthreads();
        for (int i = tid; i < 64 * 8; i += 256) {
            const int c = i >> 3, o = (i & 7) * 16;
            u32x4 vp = {0, 0, 0, 0}, vq = vp;
            const int n = wrow(c);
            if (n >= 0) vp = *(const u32x4 *)(g.w + (int64_t)n * g.K + kb * 128 + o);
            if (m0 + c < g.M) vq = *(const u32x4 *)(g.xq + (m0 + c) * g.K + kb * 128 + o);
            *(u32x4 *)&p[c][o] = vp;
            *(u32x4 *)&q[c][o] = vq;
        }
        __syncthreads();
        for (int i = 0; i < 2; ++i)
            for (int j = 0; j < 2; ++j) {
                const uint8_t *pa = &p[wp * 32 + i * 16 + (l & 15)][(l >> 4) * 32];
                const uint8_t *pb = &q[wq * 32 + j * 16 + (l & 15)][(l >> 4) * 32];
                v8i a, b;
                for (int d = 0; d < 8; ++d) {
                    a[d] = ((const int *)pa)[d];
                    b[d] = ((const int *)pb)[d];
                }
                const v4f t = mfma16x16x128(a, b);
                const int64_t m = m0 + wq * 32 + j * 16 + (l & 15);
                const float sx = m < g.M ? g.xs[m * nkb + kb] : 0.f;
                for (int v = 0; v < 4; ++v) {
                    const int n = wrow(wp * 32 + i * 16 + 4 * (l >> 4) + v);
                    if (n >= 0) acc[i][j][v] += t[v] * (sx * g.ws[(int64_t)(n >> 7) * nkb + kb]);
                }
            }
    }
    for (int j = 0; j < 2; ++j) {
        const int64_t m = m0 + wq * 32 + j * 16 + (l & 15);
        if (m >= g.M) continue;
        for (int i = 0; i < 2; ++i)
            for (int v = 0; v < 4; ++v) {
                const int n = wrow(wp * 32 + i * 16 + 4 * (l >> 4) + v);
                if (n < 0 || (sw && i == 1)) continue;
                float z = acc[i][j][v] + (g.bias ? g.bias[n] : 0.f);
                if (g.act == kActSilu) z = silu(z);
                if (g.act == kActGelu) z = gelu(z);
                if (sw) z = silu(z) * (acc[1][j][v] + (g.bias ? g.bias[n + g.n_out] : 0.f));
                if (g.res) z += bf16_bits_to_f32(g.res[m * g.ld_res + n]);
                g.out[m * g.ld_out + n] = (uint16_t)f32_to_bf16_bits(z);
            }
    }
}

}  // namespace

size_t linear_workspace(LinearArgs &, void *) { return 0; }

hipError_t launch_linear(const LinearArgs &a, hipStream_t st) {
    const int cols = a.act == kActSwiglu ? 32 : 64;
    dim3 grid((unsigned)((a.M + 63) / 64), (a.n_out + cols - 1) / cols);
    linear_kernel<<<grid, 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace moe
