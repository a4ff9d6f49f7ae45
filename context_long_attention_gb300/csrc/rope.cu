// Rotary positions of queries and keys: (a, b) -> (a cos t - b sin t,
// b cos t + a sin t) with t = position x frequency, for the pairs of the first
// or last part of every head.
//
// One pass over the rows: what bounds a prompt is reading and writing them, and
// what bounds a decode step is the chain position, angle, row, store.  So a
// thread loads its pieces of the rows first, and the angles of the block's tokens
// (one per pair, shared by all heads of a token) are made while those loads run.
//
// Angles are exact for far positions without 64-bit floating point: a frequency
// is kept as turns per position in units of 2^-64 turn, the product with the
// position wraps modulo one turn by itself in 64-bit integers, and its upper 32 bits
// are the angle, within 2^-32 turn of the given turns' (turns from frequencies in 64 bits
// are within 2^-52 of them and 2^-65 turn: at 1 radian a position 2^-24 turn at position 2^31).
// Measured: 16,384 tokens x 64 heads of 192 + 64 dims, the last 64 turned (0.8 GB)
// 119 us, all of the measured copy rate; the same in place, rotated dims alone (0.27 GB) 57;
// fp32 300 (0.8 of the rate); 64 tokens x 40 heads 4.2 us, in place 4.9.
#include <cuda_bf16.h>

#include "early_launch.cuh"
#include "internal.h"

namespace cpattn {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxAngles = 1024;  // angles of a block's tokens in shared memory

// e / d for e d < 2^32 (m = ceil(2^32 / d) passes 2^32 / d by less than 1, so
// e m / 2^32 passes e / d by less than e / 2^32 < 1 / d).
struct SmallDiv {
  uint32_t m, d;
  explicit SmallDiv(uint32_t div) : m(div > 1 ? (uint32_t)(((1ull << 32) + div - 1) / div) : 0), d(div) {}
  __device__ __forceinline__ uint32_t operator()(uint32_t e) const { return d > 1 ? __umulhi(e, m) : e; }
};

// The work on one tensor, in units of 16 elements of a head (two pieces of
// eight): its rotated pairs, eight to a unit, then the other dims where they are copied.
struct Side {
  const void* x;
  void* out;
  long long x_stride, out_stride;  // elements between tokens
  int heads, dim;
  int rot_units, units;  // of a head
  SmallDiv by_units;
  int first;             // where the rotated dims begin
  int copy_first, copy_dims;
};

struct RopeParams {
  Side s[2];
  const int32_t* pos;
  const unsigned long long* turns;  // [rot / 2]
  int T, rot;
  int tokens, splits;    // tokens that a block works on, and blocks that share them
  int token_units;       // of both tensors
  SmallDiv by_token, by_half;
  float scale, sin_scale;
};

template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 x;
  __device__ void load(const void* p, long long i) { x = __ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i)); }
  __device__ void store(void* p, long long i) const { *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) = x; }
  __device__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ void set(const float (&v)[8]) {  // rounded once, to the nearest
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    x = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Eight<float> {
  float4 x, y;
  __device__ void load(const void* p, long long i) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    x = __ldcg(q);
    y = __ldcg(q + 1);
  }
  __device__ void store(void* p, long long i) const {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = x;
    q[1] = y;
  }
  __device__ void get(float (&v)[8]) const {
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
  }
  __device__ void set(const float (&v)[8]) {
    x = make_float4(v[0], v[1], v[2], v[3]);
    y = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// N units a thread.
template <typename T, bool HALF, int N>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  __shared__ __align__(16) float s_cos[kMaxAngles], s_sin[kMaxAngles];
  wait_for_earlier_kernels();
  const int block = blockIdx.x / p.splits, part = blockIdx.x - block * p.splits;
  const int t0 = block * p.tokens, nt = min(p.tokens, p.T - t0);
  const int e0 = part * (kThreads * N) + threadIdx.x, all = nt * p.token_units;
  Eight<T> a[N], b[N];
  long long to[N] = {};  // element of the output, of the unit's first piece
  int step[N] = {};      // from the first piece to the second (0: there is none)
  int at[N];             // the unit's first angle, -1 where it is copied, -2 where there is no unit
  bool second[N] = {};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = e0 + i * kThreads;
    at[i] = -2;
    if (e >= all) continue;
    const int tok = (int)p.by_token(e);
    int u = e - tok * p.token_units;
    const int first_units = p.s[0].heads * p.s[0].units;
    second[i] = u >= first_units;
    const Side& s = p.s[second[i] ? 1 : 0];
    if (second[i]) u -= first_units;
    const int head = (int)s.by_units(u);
    u -= head * s.units;
    int d;
    if (u < s.rot_units) {
      at[i] = tok * (p.rot / 2) + 8 * u;
      d = s.first + (HALF ? 8 * u : 16 * u);
      step[i] = HALF ? p.rot / 2 : 8;
    } else {
      u = 16 * (u - s.rot_units);
      at[i] = -1;
      d = s.copy_first + u;
      step[i] = u + 8 < s.copy_dims ? 8 : 0;
    }
    const long long off = (long long)head * s.dim + d;
    const long long from = (t0 + tok) * s.x_stride + off;
    to[i] = (t0 + tok) * s.out_stride + off;
    a[i].load(s.x, from);
    if (step[i]) b[i].load(s.x, from + step[i]);
  }
  const int half = p.rot / 2;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int tok = (int)p.by_half(i);
    // the position as it is stored: a negative one turns backwards
    const unsigned long long turn = __ldcg(p.turns + (i - tok * half)) * (unsigned long long)(long long)__ldcg(p.pos + t0 + tok);
    float c, s;
    sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s, &c);
    s_cos[i] = c * p.scale;
    s_sin[i] = s * p.sin_scale;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (at[i] == -2) continue;
    void* out = p.s[second[i] ? 1 : 0].out;
    if (at[i] >= 0) {
      float x[8], y[8], c[8], s[8];
      a[i].get(x);
      b[i].get(y);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        *reinterpret_cast<float4*>(c + 4 * k) = *reinterpret_cast<const float4*>(s_cos + at[i] + 4 * k);
        *reinterpret_cast<float4*>(s + 4 * k) = *reinterpret_cast<const float4*>(s_sin + at[i] + 4 * k);
      }
      float u[8], v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // the pair: (x[k], y[k]) in halves, else neighbours 2k, 2k + 1 of the 16 elements
        const float f = HALF ? x[k] : k < 4 ? x[2 * k & 7] : y[2 * k & 7];
        const float g = HALF ? y[k] : k < 4 ? x[(2 * k & 7) + 1] : y[(2 * k & 7) + 1];
        const float r = f * c[k] - g * s[k], w = g * c[k] + f * s[k];
        if (HALF) {
          u[k] = r;
          v[k] = w;
        } else if (k < 4) {
          u[2 * k & 7] = r;
          u[(2 * k & 7) + 1] = w;
        } else {
          v[2 * k & 7] = r;
          v[(2 * k & 7) + 1] = w;
        }
      }
      a[i].set(u);
      b[i].set(v);
    }
    a[i].store(out, to[i]);
    if (step[i]) b[i].store(out, to[i] + step[i]);
  }
}

template <typename T, bool HALF>
cudaError_t launch_t(const RopeParams& p, cudaStream_t s) {
  const long long blocks = ((long long)p.T + p.tokens - 1) / p.tokens;
  const long long units = (long long)p.tokens * p.token_units;
  // One unit a thread while the blocks then fit the GPU at once, else four, whose
  // loads overlap.
  const bool one = blocks * ((units + kThreads - 1) / kThreads) <= 152 * 8;
  const long long per = (long long)kThreads * (one ? 1 : 4);
  RopeParams q = p;
  q.splits = (int)((units + per - 1) / per);
  if (blocks * q.splits > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  return launch_early(one ? rope_kernel<T, HALF, 1> : rope_kernel<T, HALF, 4>, (unsigned)(blocks * q.splits), kThreads, 0, s, 1, q);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool bf16, cudaStream_t stream) {
  auto side = [&](const RopeSide& r) {
    Side s = {r.x, r.out, r.x_stride, r.out_stride, r.heads, r.dim, a.rot / 16, 0, SmallDiv(1), 0, 0, 0};
    s.first = a.tail ? r.dim - a.rot : 0;
    s.copy_first = a.tail ? 0 : a.rot;
    s.copy_dims = r.x == r.out ? 0 : r.dim - a.rot;  // in place, the other dims are where they belong
    s.units = s.rot_units + (s.copy_dims + 15) / 16;
    s.by_units = SmallDiv((uint32_t)s.units);
    return s;
  };
  RopeParams p = {{side(a.q), side(a.k)}, a.pos, a.turns, a.T, a.rot, 1, 1, 0, SmallDiv(1), SmallDiv((uint32_t)(a.rot / 2)),
                  a.scale, a.inverse ? -a.scale : a.scale};
  p.token_units = p.s[0].heads * p.s[0].units + p.s[1].heads * p.s[1].units;
  // tokens of few units share a block
  const int most = kMaxAngles / (a.rot / 2);
  p.tokens = (4 * kThreads + p.token_units - 1) / p.token_units;
  if (p.tokens > most) p.tokens = most;
  while (p.tokens > 1 && (a.T - 1) / p.tokens < 151) p.tokens /= 2;
  p.by_token = SmallDiv((uint32_t)p.token_units);
  if (bf16) return a.half ? launch_t<__nv_bfloat16, true>(p, stream) : launch_t<__nv_bfloat16, false>(p, stream);
  return a.half ? launch_t<float, true>(p, stream) : launch_t<float, false>(p, stream);
}

}  // namespace cpattn
