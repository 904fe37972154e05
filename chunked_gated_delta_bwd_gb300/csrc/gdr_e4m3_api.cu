// C ABI of the 8-bit products (declared in include/gdr.h): argument checks and launches.
#include <limits.h>
#include <string.h>

#include "gdr_e4m3.h"
#include "gdr_host.h"

using namespace gdr;

extern "C" {

gdr_status gdr_quant_e4m3(int64_t rows, int32_t channels, const void* x, int64_t x_stride, int32_t x_type,
                          int32_t tiles, void* y, float* scale, void* y_t, float* scale_t, void* stream) {
    QuantParams p;
    memset(&p, 0, sizeof(p));
    if (rows < 0 || rows > INT_MAX) return fail(GDR_ERR_INVALID, "rows must be 0 to 2^31 - 1%s");
    if (channels < 1 || channels % 2 != 0 || channels > GDR_MAX_CHANNELS) return fail(GDR_ERR_INVALID, "channels must be even, 2 to 2^28%s");
    if (rows > ((int64_t)1 << 40) / channels) return fail(GDR_ERR_INVALID, "problem too large%s");
    if (x_type != GDR_TYPE_BF16 && x_type != GDR_TYPE_F32) return fail(GDR_ERR_UNSUPPORTED, "element types are bf16 and float32%s");
    if (x_stride == 0) x_stride = channels;
    if (x_stride < channels || x_stride % 2 != 0 || x_stride > ((int64_t)1 << 38))
        return fail(GDR_ERR_INVALID, "a row stride must be even, at least the number of channels and at most 2^38%s");
    if (!tiles && (y_t || scale_t)) return fail(GDR_ERR_INVALID, "the transposed form goes with tiles%s");
    if (!y_t != !scale_t) return fail(GDR_ERR_INVALID, "y_t and scale_t go together%s");
    if (rows == 0) return ok();
    if (!x) return fail(GDR_ERR_INVALID, "required pointer %s is NULL", "x");
    if (!aligned_to(x, x_type == GDR_TYPE_F32 ? 8 : 4)) return fail(GDR_ERR_INVALID, "pointer %s is not aligned to two elements", "x");
    NEED(y); NEED(scale); OPT(y_t); OPT(scale_t);
    const size_t codes = (size_t)rows * channels, blocks = (channels + 127) / 128;
    const size_t scales = sizeof(float) * (tiles ? ((size_t)rows + 127) / 128 : (size_t)rows) * blocks;
    const Span in[] = {{x, ((size_t)(rows - 1) * x_stride + channels) * (x_type == GDR_TYPE_F32 ? 4 : 2), "x"}};
    const Span out[] = {{y, codes, "y"}, {scale, scales, "scale"}, {y_t, codes, "y_t"}, {scale_t, scales, "scale_t"}};
    if (gdr_status st = apart(out, 4, in, 1)) return st;
    p.R = rows; p.ldx = x_stride; p.C = channels; p.x_f32 = x_type == GDR_TYPE_F32; p.tiles = tiles != 0;
    p.x = x; p.y = (uint8_t*)y; p.scale = scale; p.yt = (uint8_t*)y_t; p.scale_t = scale_t;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = timed(GDR_KERNEL_E4M3, s, [&] { return launch_quant(p, s); });
    return e == cudaSuccess ? ok() : cuda_fail(e, "quantisation launch");
}

gdr_status gdr_linear_e4m3(int64_t rows, int32_t inner, int32_t outer, const void* x, const float* x_scale,
                           int32_t x_blocks, const void* w, const float* w_scale, const float* bias, void* y,
                           void* stream) {
    LinearParams p;
    memset(&p, 0, sizeof(p));
    // (tiles of 128 rows are counted in 32 bits, from rows + 127)
    if (rows < 0 || rows > INT_MAX - 127) return fail(GDR_ERR_INVALID, "rows must be 0 to 2^31 - 128%s");
    if (inner < 1 || inner % 16 != 0 || inner > (1 << 24)) return fail(GDR_ERR_INVALID, "the inner dimension must be a multiple of 16, at most 2^24%s");
    if (outer < 1 || outer % 8 != 0 || outer > (1 << 24)) return fail(GDR_ERR_INVALID, "the outer dimension must be a multiple of 8, at most 2^24%s");
    const int blocks = (inner + 127) / 128;
    if (x_blocks != 1 && x_blocks != blocks) return fail(GDR_ERR_INVALID, "x_blocks must be 1 or ceil(inner / 128)%s");
    if (rows == 0) return ok();
    NEED(x); NEED(x_scale); NEED(w); NEED(w_scale); OPT(bias); NEED(y);
    const size_t nb = x_blocks, nk = blocks, nr = (outer + 127) / 128;
    const Span in[] = {{x, (size_t)rows * inner, "x"}, {x_scale, sizeof(float) * rows * nb, "x_scale"}, {w, (size_t)outer * inner, "w"},
                       {w_scale, sizeof(float) * nr * nk, "w_scale"}, {bias, sizeof(float) * (size_t)outer, "bias"}};
    const Span out[] = {{y, 2 * (size_t)rows * outer, "y"}};
    if (gdr_status st = apart(out, 1, in, 5)) return st;
    p.M = rows; p.K = inner; p.N = outer; p.x_blocks = x_blocks;
    p.x = (const uint8_t*)x; p.w = (const uint8_t*)w; p.xs = x_scale; p.ws = w_scale; p.bias = bias; p.y = (__nv_bfloat16*)y;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = timed(GDR_KERNEL_E4M3, s, [&] { return launch_linear(p, s); });
    return e == cudaSuccess ? ok() : cuda_fail(e, "8-bit product launch");
}

}  // extern "C"
