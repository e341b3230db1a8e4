// attention_q8.cu -- attention over the 8-bit cache, one warp per (row of q,
// query head): lane l holds elements 4 l .. 4 l + 3, keys go by one after the
// other with a running maximum and sum.
#include "pkv_device.cuh"
#include "q8.cuh"

namespace pkv {

namespace {

template <bool kE4m3>
__device__ __forceinline__ void code_values(uint32_t w, float (&x)[4]) {
  if (kE4m3) {
    const uint32_t a = e4m3x2_to_half2(w), b = e4m3x2_to_half2(w >> 16);
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(x[0]), "=f"(x[1]) : "r"(a));
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(x[2]), "=f"(x[3]) : "r"(b));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
  }
}

template <bool kE4m3>
__global__ void __launch_bounds__(256) attention_q8_kernel(const AttentionQ8Params p) {
  grid_dependency_trigger();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y;
  const int i = blockIdx.z;
  const int j = blockIdx.x * 8 + (threadIdx.x >> 5);  // row of the chunk
  const int q0 = p.cu_q != nullptr ? p.cu_q[i] : i;
  const int n = p.cu_q != nullptr ? p.cu_q[i + 1] - q0 : 1;
  if (j >= n) return;
  int ctx = p.ctx_lens[i];
  if (p.checked) {
    const bool bad = p.cu_q != nullptr ? n > p.max_q || ctx < n || ctx > p.max_context
                                       : ctx > p.max_context;
    if (bad) {
      if (lane == 0) record_error(p.err, kErrContext);
      if (p.cu_q != nullptr) return;  // the sequence is left unwritten
      ctx = p.max_context;
    }
  }
  const int seen = ctx - n + j + 1;
  const int64_t row = (static_cast<int64_t>(q0) + j) * p.Hq + h;
  const uint2 qw = *reinterpret_cast<const uint2*>(p.q + row * kHeadDim + lane * 4);
  const float q[4] = {bf16_lo(qw.x), bf16_hi(qw.x), bf16_lo(qw.y), bf16_hi(qw.y)};
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int x = 0; x < seen; ++x) {
    const int64_t block = p.tables[static_cast<int64_t>(i) * p.max_blocks + x / p.bs];
    if (p.checked && (block < 0 || block >= p.num_blocks)) {
      if (lane == 0) record_error(p.err, p.err_code);
      continue;
    }
    const int64_t r = cache_row(block, h / p.G, p.Hkv, p.bs, x % p.bs);
    const int64_t at = r * kCodeRowBytes + lane * 4;
    float k[4], v[4];
    code_values<kE4m3>(*reinterpret_cast<const uint32_t*>(p.k_codes + at), k);
    code_values<kE4m3>(*reinterpret_cast<const uint32_t*>(p.v_codes + at), v);
    float s = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= p.k_scale[r / kGroupRows] * p.qscale;
    const float mn = fmaxf(m, s);
    const float a = fast_exp2(m - mn), w = fast_exp2(s - mn);
    const float wv = w * p.v_scale[r / kGroupRows];
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = o[e] * a + wv * v[e];
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  *reinterpret_cast<uint2*>(p.out + row * kHeadDim + lane * 4) =
      make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
}

}  // namespace

cudaError_t launch_attention_q8(const AttentionQ8Params& p, bool e4m3, cudaStream_t stream) {
  const dim3 grid((p.max_q + 7) / 8, p.Hq, p.num_seqs);
  return e4m3 ? launch_pdl(attention_q8_kernel<true>, grid, dim3(256), 0, stream, p)
              : launch_pdl(attention_q8_kernel<false>, grid, dim3(256), 0, stream, p);
}

}  // namespace pkv
