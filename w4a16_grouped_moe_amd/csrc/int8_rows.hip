// Symmetric 8-bit quantisation of rows, one fp32 scale each (the arithmetic:
// int8_quant.hpp). A wave takes a row; with few rows a whole workgroup does.
//
// Bound by reading x and writing q once: the row stays in registers between
// its maximum and its codes. 16001 rows of 2803 bf16: 28.3 us (4.75 TB/s; a
// large device copy moves 4.8 to 5.2 on the same card); 256 rows of 2816 fp16:
// 3.8 us, most of it the launch (5.3 with a wave per row).
#include "int8_common.hpp"
#include "int8_quant.hpp"

namespace dgw4 {
namespace {

constexpr int kRowThreads = 512;

template <class Tx>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const Tx *__restrict__ x, int rows, int K,
                                                            long long ldx, int8_t *__restrict__ q, long long ldq,
                                                            float *__restrict__ s)
{
    const int lane = threadIdx.x & 63;
    const size_t row = (size_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= (size_t)rows)
        return;
    const float sc = quantize_row<Tx, 64, 6>(x + row * ldx, K, (K + 15) / 16 * 16, (char *)q + row * ldq, lane, nullptr);
    if (lane == 0)
        s[row] = sc;
}

template <class Tx>
__global__ void __launch_bounds__(kRowThreads) quantize_row_kernel(const Tx *__restrict__ x, int K, long long ldx,
                                                                   int8_t *__restrict__ q, long long ldq,
                                                                   float *__restrict__ s)
{
    __shared__ uint32_t s_part[kRowThreads / 64];
    const size_t row = blockIdx.x;
    const float sc = quantize_row<Tx, kRowThreads, 2>(x + row * ldx, K, (K + 15) / 16 * 16, (char *)q + row * ldq,
                                                      threadIdx.x, s_part);
    if (threadIdx.x == 0)
        s[row] = sc;
}

template <class Tx>
hipError_t run(const void *x, int rows, int K, long long ldx, int8_t *q, long long ldq, float *s, hipStream_t st)
{
    // a wave per row needs a thousand rows to fill the chip
    if (rows < 1024 && K > 1024)
        quantize_row_kernel<Tx><<<dim3(rows), dim3(kRowThreads), 0, st>>>((const Tx *)x, K, ldx, q, ldq, s);
    else
        quantize_rows_kernel<Tx>
            <<<dim3(((unsigned)rows + 3) / 4), dim3(256), 0, st>>>((const Tx *)x, rows, K, ldx, q, ldq, s);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows(const void *x, int type, int rows, int K, long long ldx, int8_t *q,
                                long long ldq, float *s, hipStream_t stream)
{
    return type == DGW4_F32   ? run<float>(x, rows, K, ldx, q, ldq, s, stream)
           : type == DGW4_F16 ? run<_Float16>(x, rows, K, ldx, q, ldq, s, stream)
                              : run<__bf16>(x, rows, K, ldx, q, ldq, s, stream);
}

}  // namespace dgw4
