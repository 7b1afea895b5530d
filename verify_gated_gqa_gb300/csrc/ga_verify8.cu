// Decode and verify attention over 8-bit paged caches (format: ga_q8.cuh).
//
// Per sequence with L cached tokens before the window, window row r (position L + r) sees keys
// 0 .. L + r; with s_j = q . k_j / 16, out = (sum_j e^(s_j) v_j / sum_j e^(s_j)) sigmoid(gate).
//
// A CTA runs one (row, KV head) with its 12 query heads over all keys, a block of 32 keys at a time:
// a warp forms the scores of four keys, then each thread keeps one dim of O for the 12 heads.
#include "ga_q8.cuh"
#include "ga_v4.cuh"

namespace ga {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2eOver16 = 1.4426950408889634f / 16.0f;

__global__ void __launch_bounds__(kThreads) verify8_kernel(const __grid_constant__ Verify8Args a) {
  __shared__ float q[kGroup][kDim], w[kGroup][kQ8Block], M[kGroup], l[kGroup], scale[kGroup];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / a.rows, r = blockIdx.x - b * a.rows, head = blockIdx.y;
  const int L = a.seq_len[b];
  const long long keys_all = (long long)L + a.rows;
  if (L < 0) return;
  if (keys_all > (long long)a.max_pages * a.page_size || keys_all > GA_MAX_TOKENS) {
    if (tid == 0) record(a.status, kDevBadPosition);
    return;
  }
  const size_t row = ((size_t)b * a.rows + r) * kHeads + head * kGroup;
  for (int i = tid; i < kGroup * kDim; i += kThreads)
    q[i / kDim][i % kDim] = lo_f(a.q_prep[row * kDim + i]);
  if (tid < kGroup) {
    M[tid] = -INFINITY;
    l[tid] = 0.f;
  }
  float o[kGroup];
  for (int h = 0; h < kGroup; ++h) o[h] = 0.f;
  const int keys = L + r + 1;
  for (int key0 = 0; key0 < keys; key0 += kQ8Block) {
    const int e = key0 / a.page_size, page = a.page_table[(size_t)b * a.max_pages + e];
    const bool good = page >= 0 && page < a.n_pages;
    if (!good && tid == 0) record(a.status, kDevBadPage);
    const size_t at = ((size_t)(good ? page : 0) * kKvHeads + head) * a.page_size + key0 - e * a.page_size;
    const float ks = good ? pow2i(q8_exp(a.k_scales[at / kQ8Block])) : 0.f;
    const float vs = good ? pow2i(q8_exp(a.v_scales[at / kQ8Block])) : 0.f;
    __syncthreads();
    for (int j = 4 * warp; j < 4 * warp + 4; ++j) {
      const bool seen = key0 + j < keys;
      float k[8];
      for (int d = 0; d < 8; ++d)
        k[d] = seen && good ? f16x2_f32(e4m3x2_f16x2(a.k_codes[(at + j) * kDim + 8 * lane + d])).x : 0.f;
      for (int h = 0; h < kGroup; ++h) {
        float s = 0.f;
        for (int d = 0; d < 8; ++d) s += q[h][8 * lane + d] * k[d];
        for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(~0u, s, off);
        if (lane == 0) w[h][j] = seen ? s * ks * kLog2eOver16 : -INFINITY;
      }
    }
    __syncthreads();
    if (tid < kGroup) {
      float top = M[tid];
      for (int j = 0; j < kQ8Block; ++j) top = fmaxf(top, w[tid][j]);
      scale[tid] = exp2f(M[tid] - top);
      float sum = l[tid] * scale[tid];
      for (int j = 0; j < kQ8Block; ++j) sum += w[tid][j] = exp2f(w[tid][j] - top);
      M[tid] = top;
      l[tid] = sum;
    }
    __syncthreads();
    for (int h = 0; h < kGroup; ++h) o[h] *= scale[h];
    for (int j = 0; j < min(kQ8Block, keys - key0); ++j) {
      const float v = good ? f16x2_f32(e4m3x2_f16x2(a.v_codes[(at + j) * kDim + tid])).x * vs : 0.f;
      for (int h = 0; h < kGroup; ++h) o[h] += w[h][j] * v;
    }
  }
  for (int h = 0; h < kGroup; ++h) {
    const float g = lo_f(a.qg[(row + h) * kQgStride + kDim + tid]);
    a.out[(row + h) * kDim + tid] = (uint16_t)(pack_bf16x2(o[h] / l[h] * sigmoid_f(g), 0.f) & 0xFFFFu);
  }
}

}  // namespace

cudaError_t launch_verify8(const Verify8Args& a, cudaStream_t s) {
  verify8_kernel<<<dim3((unsigned)(a.n_seq * a.rows), kKvHeads), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ga
