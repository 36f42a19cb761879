// Symmetric 8-bit quantisation of rows, one fp32 scale each (the arithmetic:
// int8_quant.hpp). A row belongs to 8 to 64 lanes of a wave, or to a workgroup,
// by its length.
//
// Bound by reading x and writing q once: the row stays in registers between
// its maximum and its codes (up to 16384 columns). 16001 rows of 2803 bf16: 24.3
// us (5.5 TB/s; a large device copy moves 4.8 to 5.2 on the same card); 65536
// rows of 64 fp16 5.8 us (a wave per row: 37), 2700 of 16384 bf16 31 (a wave per
// row, which reads x twice: 53); 256 rows of 2816 fp16 3.3 us, most of it the
// launch.
#include "int8_common.hpp"
#include "int8_quant.hpp"

namespace dgw4 {
namespace {

// N lanes of a wave take a row.
template <class Tx, int N, int kKept>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const Tx *__restrict__ x, int rows, int K,
                                                            long long ldx, int8_t *__restrict__ q, long long ldq,
                                                            float *__restrict__ s)
{
    const int lane = threadIdx.x % N;
    const size_t row = (size_t)blockIdx.x * (256 / N) + threadIdx.x / N;
    if (row >= (size_t)rows)
        return;
    const float sc = quantize_row<Tx, N, kKept>(x + row * ldx, K, (K + 15) / 16 * 16, (char *)q + row * ldq, lane, nullptr);
    if (lane == 0)
        s[row] = sc;
}

// A workgroup of N threads takes a row.
template <class Tx, int N, int kKept>
__global__ void __launch_bounds__(N) quantize_row_kernel(const Tx *__restrict__ x, int K, long long ldx,
                                                         int8_t *__restrict__ q, long long ldq, float *__restrict__ s)
{
    __shared__ uint32_t s_part[N / 64];
    const size_t row = blockIdx.x;
    const float sc = quantize_row<Tx, N, kKept>(x + row * ldx, K, (K + 15) / 16 * 16, (char *)q + row * ldq,
                                                threadIdx.x, s_part);
    if (threadIdx.x == 0)
        s[row] = sc;
}

// In as many launches as keep one under 2^30 threads (2^32 are refused).
template <class Tx, int N, int kKept>
void rows_in(const void *x, int rows, int K, long long ldx, int8_t *q, long long ldq, float *s, hipStream_t st)
{
    constexpr int most = (1 << 30) / N;
    for (long long at = 0; at < rows; at += most) {
        const int n = (int)(rows - at < most ? rows - at : most);
        const Tx *xa = static_cast<const Tx *>(x) + at * ldx;
        if constexpr (N <= 64)
            quantize_rows_kernel<Tx, N, kKept><<<dim3((n - 1) / (256 / N) + 1), dim3(256), 0, st>>>(
                xa, n, K, ldx, q + at * ldq, ldq, s + at);
        else
            quantize_row_kernel<Tx, N, kKept><<<dim3(n), dim3(N), 0, st>>>(xa, K, ldx, q + at * ldq, ldq, s + at);
    }
}

template <class Tx>
hipError_t run(const void *x, int rows, int K, long long ldx, int8_t *q, long long ldq, float *s, hipStream_t st)
{
    // The least room for K, and then few vectors a thread: a lane's loads past
    // the row are issued all the same. Many rows of some 2000 to 2800 stay with
    // a wave each (16001 x 2803 bf16 in a graph 30 us, 34 with 256 threads;
    // 3000 x 2816 fp16 10.6 and 9.8).
    if (K <= 128)
        rows_in<Tx, 8, 2>(x, rows, K, ldx, q, ldq, s, st);
    else if (K <= 384)
        rows_in<Tx, 16, 3>(x, rows, K, ldx, q, ldq, s, st);
    else if (K <= 768)
        rows_in<Tx, 32, 3>(x, rows, K, ldx, q, ldq, s, st);
    else if (K <= 1024)
        rows_in<Tx, 64, 2>(x, rows, K, ldx, q, ldq, s, st);
    else if (K <= 1536)
        rows_in<Tx, 32, 6>(x, rows, K, ldx, q, ldq, s, st);
    else if (K <= 64 * 48 && rows >= 8192)
        rows_in<Tx, 64, 6>(x, rows, K, ldx, q, ldq, s, st);
    else if (K <= 4096)
        rows_in<Tx, 256, 2>(x, rows, K, ldx, q, ldq, s, st);
    else if (K <= 8192)
        rows_in<Tx, 512, 2>(x, rows, K, ldx, q, ldq, s, st);
    else
        rows_in<Tx, 512, 4>(x, rows, K, ldx, q, ldq, s, st);
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
