// Attention over the paged cache in full precision (fp32 pools): one warp per new token and head.
#include "cache_row.cuh"

namespace pisa {
namespace cache {
namespace {

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(kWarps * 32) attn_simt(const AttnArgs a) {
  constexpr int kCols = D / 32;
  __shared__ float qs[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
  Seq s;
  if (!load_seq(a.seqs, b, a.q.rows, &s)) return;
  const long long row = (long long)blockIdx.x * kWarps + warp;
  const int i = (int)(row / a.heads), h = (int)(row % a.heads);
  if (i >= s.n) return;
  const long long qi = s.row0 + i;
  const float* q = reinterpret_cast<const float*>(a.q.data + b * a.q.seq + qi * a.q.row + (long long)h * a.q.head);
  for (int c = lane; c < D; c += 32) qs[warp][c] = q[c];
  __syncwarp();
  int first, last;
  visible(a, s.len, s.len - s.n + i, &first, &last);
  float m, l, acc[kCols];
  row_attention<float, D>(a, b, h / a.group, qs[warp], first, last, &m, &l, acc);
  float* o = reinterpret_cast<float*>(a.o.data + b * a.o.seq + qi * a.o.row + (long long)h * a.o.head);
  const float inv = l == 0.f ? 0.f : 1.f / l;      // NaN sums stay NaN
#pragma unroll
  for (int c = 0; c < kCols; ++c) o[c * 32 + lane] = acc[c] * inv;
  float* lse = lse_at(a, b, s, i, h);
  if (lse && lane == 0) *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
  const long long blocks = ((long long)a.seqs.max_new * a.heads + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  attn_simt<D><<<dim3((unsigned)blocks, a.seqs.batch), kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_simt(const AttnArgs& a, int d, cudaStream_t st) {
  return d == 64 ? launch<64>(a, st) : launch<128>(a, st);
}

}  // namespace cache
}  // namespace pisa
