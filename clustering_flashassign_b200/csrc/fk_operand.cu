// Operand copies of the soft assignment products.
#include "fk_logprob.cuh"

namespace fk {
namespace soft {
namespace {

// Operand copies: 16-bit rows as they are, fp32 rows as three bf16 planes of
// dp >= d elements (zero padded).  drop: rows whose gradient is zero whatever
// they hold (padding), or table rows that a bias of -inf masks, become zero,
// so that what they hold (NaN included) stays out of the products.
template <typename T>
__global__ void __launch_bounds__(256)
    k_operand(const T *src, long long rows, long long rows_per_b, int d, int dp, const RowGrad *grads,
              const float *bias, void *dst) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= rows) return;
  const bool drop = (grads && grads[r].id == -2) || (bias && bias[r] == kNegInf);
  const T *in = src + (size_t)r * d;
  if constexpr (sizeof(T) == 2) {
    uint4 *out = reinterpret_cast<uint4 *>(static_cast<T *>(dst) + (size_t)r * d);
    for (int j = lane; j < d / 8; j += 32)
      out[j] = drop ? make_uint4(0, 0, 0, 0) : __ldg(reinterpret_cast<const uint4 *>(in) + j);
  } else {
    const long long b = r / rows_per_b;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(dst) + ((size_t)(b * 3) * rows_per_b + (r - b * rows_per_b)) * dp;
    const size_t plane = (size_t)rows_per_b * dp;
    for (int j = lane; j < dp; j += 32) {
      float v = j < d && !drop ? in[j] : 0.f;
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        out[p * plane + j] = h;
        // an infinity (or an overflow of the rounding) leaves no remainder
        const float rest = v - __bfloat162float(h);
        v = fabsf(__bfloat162float(h)) < INFINITY ? rest : 0.f;
      }
    }
  }
}

template <typename T>
int launch_operand(const void *src, long long rows, long long rows_per_b, int d, int dp, const RowGrad *g,
                   const float *bias, void *dst, cudaStream_t s) {
  FK_CUDA(launch_pdl(k_operand<T>, dim3((unsigned)cdiv(rows, 8)), dim3(256), 0, s, static_cast<const T *>(src), rows,
                     rows_per_b, d, dp, g, bias, dst));
  return launched();
}

}  // namespace

int operand(const void *src, int dtype, long long rows, long long rows_per_b, int d, int dp, const RowGrad *g,
            const float *bias, void *dst, cudaStream_t s) {
  if (dtype == FK_F32) return launch_operand<float>(src, rows, rows_per_b, d, dp, g, bias, dst, s);
  return launch_operand<__half>(src, rows, rows_per_b, d, dp, g, bias, dst, s);  // 16-bit rows are copied as bits
}

}  // namespace soft
}  // namespace fk
