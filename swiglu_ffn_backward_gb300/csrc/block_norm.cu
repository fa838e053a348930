// The junction of two blocks of a transformer: the norm after a block, its gate, the scaled residual, and the norm
// before the next block (root mean square norms, over the last dimension), forward and backward.
//   rstd(t) = 1 / sqrt(sum t^2 / N + eps)
//   v = u rstd(u) gamma_post  (v = u without the norm after the block)
//   h = alpha r + gate v, rounded to the I/O type;  y = h rstd(h) gamma_pre
// A row of the gate serves M / G rows, one after the other. Backward, with u^ = u rstd(u), h^ = h rstd(h),
// a = dy gamma_pre and q = gate gamma_post, from dy and dh, the gradient that reaches h past the second norm:
//   D  = dh + rstd(h) (a - h^ mean(a h^)),  dr = alpha D
//   du = rstd(u) (q D - u^ mean(q D u^))
//   dgamma_pre = sum dy h^;  with S = sum D u^ over the rows of a gate row: dgate = gamma_post S, and
//   dgamma_post = the sum of gate S over the gate's rows
// so that two column sums give all three parameter gradients. The second mean needs no second round over the row:
//   sum q D u^ = sum q u^ (dh + rstd(h) a) - rstd(h) mean(a h^) sum q h^ u^
// All arithmetic is fp32; h, y, dr, du and the parameters' gradients are rounded once.
#include <algorithm>

#include "row_vectors.cuh"

namespace swg {
namespace {

using namespace row;

constexpr int kMaxThreads = 1024;

// ---- rows of any length, element by element, read three times (from L2 where a row fits)
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) bn_fwd_long_kernel(const BnFwdArgs a) {
  __shared__ float buf[32];
  const float inv_n = 1.0f / static_cast<float>(a.N);
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    const T* u = static_cast<const T*>(a.u) + r * a.ldu;
    const T* res = a.residual != nullptr ? static_cast<const T*>(a.residual) + r * a.ldr : nullptr;
    const int64_t gate = r / a.rows_per_gate * a.N;
    T* h = a.h != nullptr ? static_cast<T*>(a.h) + r * a.N : nullptr;
    float s[1], ru = 0.0f, rh = 0.0f;
    if (a.post) {
      long_sums(a.N, s, [&](float (&p)[1], int64_t j) {
        const float v = to_f(u[j]);
        p[0] = fmaf(v, v, p[0]);
      });
      ru = rsqrtf(fmaf(block_sum(s[0], buf), inv_n, a.eps));
    }
    auto value = [&](int64_t j) {  // h_j, rounded as it is stored
      if (a.h == nullptr) return to_f(u[j]);
      float v = to_f(u[j]);
      if (a.post) v *= ru * (a.gamma_post != nullptr ? load_any(a.gamma_post, j, a.wdtype) : 1.0f);
      if (a.gate != nullptr) v *= load_any(a.gate, gate + j, a.gdtype);
      if (res != nullptr) v = fmaf(a.alpha, to_f(res[j]), v);
      return to_f(from_f<T>(v));
    };
    if (a.pre) {
      long_sums(a.N, s, [&](float (&p)[1], int64_t j) {
        const float v = value(j);
        p[0] = fmaf(v, v, p[0]);
      });
      rh = rsqrtf(fmaf(block_sum(s[0], buf), inv_n, a.eps));
    }
    for (int64_t j = threadIdx.x; j < a.N; j += blockDim.x) {
      const float v = value(j);
      if (h != nullptr) h[j] = from_f<T>(v);
      if (a.pre)
        static_cast<T*>(a.y)[r * a.N + j] =
            from_f<T>(v * (rh * (a.gamma_pre != nullptr ? load_any(a.gamma_pre, j, a.wdtype) : 1.0f)));
    }
    if (threadIdx.x == 0) {
      a.stats[2 * r] = ru;
      a.stats[2 * r + 1] = rh;
    }
  }
}

// What belongs to element j of row r in the backward. u^ is u where there is no norm after the block.
template <typename T>
struct Element {
  float uh, hh, a, dh, q, gate, post;
  __device__ __forceinline__ Element(const BnBwdArgs& p, int64_t r, int64_t j, float ru, float rh) {
    uh = to_f(static_cast<const T*>(p.u)[r * p.ldu + j]) * (p.post ? ru : 1.0f);
    hh = p.pre ? to_f(static_cast<const T*>(p.h)[r * p.ldh + j]) * rh : 0.0f;
    a = p.pre ? to_f(static_cast<const T*>(p.dy)[r * p.lddy + j]) : 0.0f;  // dy; times gamma_pre below
    dh = p.dh != nullptr ? to_f(static_cast<const T*>(p.dh)[r * p.lddh + j]) : 0.0f;
    post = p.post && p.gamma_post != nullptr ? load_any(p.gamma_post, j, p.wdtype) : 1.0f;
    gate = p.gate != nullptr ? load_any(p.gate, r / p.rows_per_gate * p.N + j, p.gdtype) : 1.0f;
    q = gate * post;
  }
};
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) bn_dx_long_kernel(const BnBwdArgs a) {
  __shared__ float buf[32];
  const float inv_n = 1.0f / static_cast<float>(a.N);
  const bool rows_gate = a.dgate != nullptr && a.rows_per_gate == 1;
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    const float ru = a.post ? a.stats[2 * r] : 0.0f, rh = a.pre ? a.stats[2 * r + 1] : 0.0f;
    auto pre = [&](int64_t j) { return a.pre && a.gamma_pre != nullptr ? load_any(a.gamma_pre, j, a.wdtype) : 1.0f; };
    float s[3];
    long_sums(a.N, s, [&](float (&p)[3], int64_t j) {
      const Element<T> e(a, r, j, ru, rh);
      const float g = e.a * pre(j), qu = e.q * e.uh;
      p[0] = fmaf(g, e.hh, p[0]);
      p[1] = fmaf(qu, fmaf(rh, g, e.dh), p[1]);
      p[2] = fmaf(qu, e.hh, p[2]);
    });
    const float c1 = block_sum(s[0], buf) * inv_n * rh, s1 = block_sum(s[1], buf), s2 = block_sum(s[2], buf);
    const float c2 = a.post ? fmaf(-c1, s2, s1) * inv_n : 0.0f;
    for (int64_t j = threadIdx.x; j < a.N; j += blockDim.x) {
      const Element<T> e(a, r, j, ru, rh);
      const float d = fmaf(rh, e.a * pre(j), fmaf(-c1, e.hh, e.dh));
      if (a.dres != nullptr) static_cast<T*>(a.dres)[r * a.N + j] = from_f<T>(a.alpha * d);
      const float du = a.post ? ru * fmaf(-e.uh, c2, e.q * d) : e.q * d;
      static_cast<T*>(a.du)[r * a.N + j] = from_f<T>(du);
      if (rows_gate) store_any(a.dgate, r * a.N + j, a.gdtype, d * e.uh * e.post);
    }
    if (threadIdx.x == 0 && a.mean != nullptr) a.mean[r] = c1;
  }
}

// One chunk's column sums, for rows of any length: part[chunk][0][j] of D u^ (times the gate where it has a row for
// each row), part[chunk][1][j] of dy h^.
constexpr int kColThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kColThreads) bn_param_long_kernel(const BnBwdArgs a, const BnChunks k, int64_t first) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kColThreads + threadIdx.x, chunk = first + blockIdx.y;
  if (j >= a.N) return;
  const int64_t seg = chunk / k.per_segment, r0 = seg * k.segment + chunk % k.per_segment * k.rows;
  const int64_t r1 = min((seg + 1) * k.segment, r0 + k.rows);
  const float pre = a.pre && a.gamma_pre != nullptr ? load_any(a.gamma_pre, j, a.wdtype) : 1.0f;
  float s = 0.0f, p = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
    const float ru = a.post ? a.stats[2 * r] : 0.0f, rh = a.pre ? a.stats[2 * r + 1] : 0.0f;
    const Element<T> e(a, r, j, ru, rh);
    const float d = fmaf(rh, e.a * pre, fmaf(-a.mean[r], e.hh, e.dh));
    s = fmaf(d * e.uh, a.rows_per_gate == 1 ? e.gate : 1.0f, s);
    p = fmaf(e.a, e.hh, p);
  }
  float* to = a.part + chunk * 2 * a.N;
  to[j] = s;
  to[a.N + j] = p;
}

// The parameters' gradients from the chunks' sums: 32 columns a block, sixteen threads a column take the chunks in
// turn and are added in order. Blocks of the first row sum all chunks, for dgamma_post (each times its gate row) and
// dgamma_pre; those of row 1 + g the chunks of gate row g. 64 terms are added in fp32, these parts in fp64.
constexpr int kReduceCols = 32, kReduceSlices = 16;
__global__ void __launch_bounds__(kReduceCols* kReduceSlices)
    bn_reduce_kernel(const BnBwdArgs a, const BnChunks k, int64_t first_gate, bool sums) {
  __shared__ double acc[kReduceSlices][kReduceCols];
  const int c = threadIdx.x % kReduceCols, slice = threadIdx.x / kReduceCols;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kReduceCols + c;
  const bool whole = sums && blockIdx.y == 0;  // over all chunks
  const int64_t g = first_gate + blockIdx.y - (sums ? 1 : 0);
  const int64_t begin = whole ? 0 : g * k.per_segment, end = whole ? k.chunks : begin + k.per_segment;
  const bool weigh = whole && a.gate != nullptr && a.rows_per_gate > 1 && j < a.N;
  const int64_t most = whole ? 2 * a.N : a.N;
  double t = 0.0;
  if (j < most) {
    for (int64_t i = begin + slice; i < end; i += 64 * kReduceSlices) {
      float s = 0.0f;
      const int64_t stop = min(end, i + 64 * kReduceSlices);
      for (int64_t n = i; n < stop; n += kReduceSlices) {
        const float v = a.part[n * 2 * a.N + j];
        s = weigh ? fmaf(v, load_any(a.gate, n / k.per_segment * a.N + j, a.gdtype), s) : s + v;
      }
      t += static_cast<double>(s);
    }
  }
  acc[slice][c] = t;
  __syncthreads();
  if (slice != 0 || j >= most) return;
  for (int i = 1; i < kReduceSlices; ++i) t += acc[i][c];
  const float v = static_cast<float>(t);
  if (!whole) {
    const float post = a.post && a.gamma_post != nullptr ? load_any(a.gamma_post, j, a.wdtype) : 1.0f;
    store_any(a.dgate, g * a.N + j, a.gdtype, v * post);
  } else if (j < a.N) {
    if (a.dgamma_post != nullptr) store_any(a.dgamma_post, j, a.wdtype, v);
  } else if (a.dgamma_pre != nullptr) {
    store_any(a.dgamma_pre, j - a.N, a.wdtype, v);
  }
}

// ---- host
// Chunks of rows whose column sums are taken together: of one gate row where the gate has fewer rows than M, and of
// at most 128 rows (like terms are rounded the same way, and a longer chain drifts).
constexpr int64_t kMostRows = 128, kLongChunks = 304;
BnChunks chunks_of(int64_t M, int64_t rows_per_gate, int64_t wanted) {
  BnChunks k;
  k.segment = rows_per_gate > 1 ? rows_per_gate : M;
  const int64_t segments = M / k.segment;
  k.rows = std::min<int64_t>(kMostRows, std::max<int64_t>(1, (M + wanted - 1) / wanted));
  k.per_segment = (k.segment + k.rows - 1) / k.rows;
  k.chunks = segments * k.per_segment;
  return k;
}

cudaError_t launch_reduce(const BnBwdArgs& a, const BnChunks& k, cudaStream_t stream) {
  const bool sums = a.dgamma_post != nullptr || a.dgamma_pre != nullptr;
  const int64_t gates = a.dgate != nullptr && a.rows_per_gate > 1 ? a.M / a.rows_per_gate : 0;
  const int64_t all = gates + (sums ? 1 : 0);
  const unsigned gx = static_cast<unsigned>(((sums ? 2 : 1) * a.N + kReduceCols - 1) / kReduceCols);
  for (int64_t y = 0; y < all; y += 65535) {
    const bool first = sums && y == 0;
    const dim3 grid(gx, static_cast<unsigned>(std::min<int64_t>(65535, all - y)));
    bn_reduce_kernel<<<grid, kReduceCols * kReduceSlices, 0, stream>>>(a, k, first ? 0 : y - (sums ? 1 : 0), first);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T>
cudaError_t fwd_type(const BnFwdArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.M, 65536));
  bn_fwd_long_kernel<T><<<grid, kMaxThreads, 0, stream>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t bwd_type(const BnBwdArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.M, 65536));
  bn_dx_long_kernel<T><<<grid, kMaxThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.part == nullptr) return e;
  const BnChunks k = chunks_of(a.M, a.rows_per_gate, kLongChunks);
  for (int64_t c = 0; c < k.chunks; c += 65535) {
    const dim3 g(static_cast<unsigned>((a.N + kColThreads - 1) / kColThreads),
                 static_cast<unsigned>(std::min<int64_t>(65535, k.chunks - c)));
    bn_param_long_kernel<T><<<g, kColThreads, 0, stream>>>(a, k, c);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return launch_reduce(a, k, stream);
}

}  // namespace

size_t bn_workspace_bytes(int64_t M, int64_t N, int64_t rows_per_gate) {
  const BnChunks k = chunks_of(M, rows_per_gate, kLongChunks);
  return (static_cast<size_t>(k.chunks) * 2 * N + M) * sizeof(float);
}

cudaError_t launch_block_norm_fwd(const BnFwdArgs& a, int dtype, cudaStream_t stream) {
  return dtype == 0   ? fwd_type<float>(a, stream)
         : dtype == 1 ? fwd_type<__half>(a, stream)
                      : fwd_type<__nv_bfloat16>(a, stream);
}

cudaError_t launch_block_norm_bwd(const BnBwdArgs& given, void* workspace, int dtype, cudaStream_t stream) {
  BnBwdArgs a = given;
  if (workspace != nullptr) {  // the rows' means, then the chunks' sums
    a.part = static_cast<float*>(workspace);
    a.mean = a.part + chunks_of(a.M, a.rows_per_gate, kLongChunks).chunks * 2 * a.N;
  }
  return dtype == 0   ? bwd_type<float>(a, stream)
         : dtype == 1 ? bwd_type<__half>(a, stream)
                      : bwd_type<__nv_bfloat16>(a, stream);
}

}  // namespace swg
