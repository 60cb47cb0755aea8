// rotate.cu -- dspark_rope_table (host), dspark_qk_rotate, dspark_rotate_write
// and dspark_latent_write: norms and position rotations between the
// projections of a step and its attention.
#define DSPARK_TU 15  // this file's number in the checked build's site codes

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "common.cuh"

namespace dspark {

// ------------------------------------------------------------- frequencies
// A frequency is kept as turns per position in 0.64 fixed point: position *
// turns modulo 2^64 is then the angle, exact however far the position is
// (an fp32 product is off by 2^-24 of the angle, 0.06 radians at 10^6).
void rope_table(int rot_dim, double base, int scaling, double factor, double original_len,
                double low, double high, const double* inv_freq, uint64_t* table) {
  const double tau = 6.283185307179586476925286766559;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = inv_freq ? inv_freq[i] : std::pow(base, -2.0 * i / rot_dim);
    if (scaling == DSPARK_ROPE_LINEAR) f /= factor;
    if (scaling == DSPARK_ROPE_PARTS) {
      const double turns = original_len * f / tau;  // over the original length
      double keep = (turns - low) / (high - low);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      f *= keep + (1.0 - keep) / factor;
    }
    const double turn = f / tau;
    // modulo one turn; below 2^-64 of one nothing is left
    const double part = turn - std::floor(turn);
    const double scaled = std::nearbyint(std::ldexp(part, 64));
    table[i] = scaled >= 18446744073709551616.0 ? 0u : (uint64_t)scaled;
  }
}

namespace {

constexpr int kRotThreads = 256;
constexpr int kRotTokens = 4;  // of a CTA, 64 threads each
constexpr int kRotLanes = kRotThreads / kRotTokens;
constexpr int kMaxRot = 256;

struct RotateParams {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_token, q_head, k_token, k_head;  // elements, as all strides
  int n_src, n_tokens;
  int heads, kv_heads, rows;  // rows: of a token, queries then keys then values
  int dim, lane_bits;         // lanes of a row: a power of two of at least dim / 8
  const float* q_weight;
  const float* k_weight;
  float eps;
  const int32_t* positions;
  const uint64_t* table;
  int rot_start, rot_dim;
  float magnitude;
  void* q_out;
  int64_t qo_token, qo_head;
  void* k_out;   // the keys' outputs, or the key cache
  void* v_out;   // the value cache
  int64_t ko_token, ko_head;
  int64_t block_stride;
  int n_blocks, page;
  const int32_t* slots;  // NULL: no cache
  const int32_t* src_rows;
  int per;  // rows of a token that one CTA takes
};

// four elements in memory, and as floats
template <typename T>
struct Quad {
  using Load = uint2;
  static __device__ __forceinline__ float4 widen(uint2 w) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>)
      return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                         __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
    return make_float4(a.x, a.y, b.x, b.y);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint2 round(float4 f) {
    return make_uint2(pack(f.x, f.y), pack(f.z, f.w));
  }
};
template <>
struct Quad<float> {
  using Load = float4;
  static __device__ __forceinline__ float4 widen(float4 f) { return f; }
  static __device__ __forceinline__ float4 round(float4 f) { return f; }
};

// cos and sin of `position` times a table entry, times the magnitude.  The
// angle as a signed fraction of a half turn is rounded to fp32 once: off by
// 2^-25 pi at most.
__device__ __forceinline__ float2 turn_of(int position, uint64_t turns, float magnitude) {
  float s, c;
  const int64_t angle = (int64_t)((uint64_t)(uint32_t)position * turns);
  sincospif((float)angle * 0x1p-63f, &s, &c);
  return make_float2(c * magnitude, s * magnitude);
}

__device__ __forceinline__ float4 scale4(float4 x, float f, float4 w) {
  return make_float4(x.x * f * w.x, x.y * f * w.y, x.z * f * w.z, x.w * f * w.w);
}

// the pairs of (a, b) turned: in the half layout a's elements with b's, in
// the interleaved one neighbours
template <bool kInterleaved>
__device__ __forceinline__ void turn8(float4& a, float4& b, const float (&c)[4],
                                      const float (&s)[4]) {
  const float4 x = a, y = b;
  if constexpr (kInterleaved) {
    a = make_float4(x.x * c[0] - x.y * s[0], x.y * c[0] + x.x * s[0], x.z * c[1] - x.w * s[1],
                    x.w * c[1] + x.z * s[1]);
    b = make_float4(y.x * c[2] - y.y * s[2], y.y * c[2] + y.x * s[2], y.z * c[3] - y.w * s[3],
                    y.w * c[3] + y.z * s[3]);
  } else {
    a = make_float4(x.x * c[0] - y.x * s[0], x.y * c[1] - y.y * s[1], x.z * c[2] - y.z * s[2],
                    x.w * c[3] - y.w * s[3]);
    b = make_float4(y.x * c[0] + x.x * s[0], y.y * c[1] + x.y * s[1], y.z * c[2] + x.z * s[2],
                    y.w * c[3] + x.w * s[3]);
  }
}

// Where a lane's eight elements lie in a head's row: two fours.  A lane of
// the rotated part has four whole pairs, so nothing is exchanged between
// lanes: in the half layout the fours are rot_dim / 2 apart.
struct Place {
  int a, b;
  int pair;  // the first of its pairs, -1 outside the rotated part
};
template <bool kInterleaved>
__device__ __forceinline__ Place place_of(int lane, int rot_start, int rot_dim) {
  const int j = lane - rot_start / 8;
  if (j < 0 || j >= rot_dim / 8) return {lane * 8, lane * 8 + 4, -1};
  if (kInterleaved) return {lane * 8, lane * 8 + 4, 4 * j};
  return {rot_start + 4 * j, rot_start + rot_dim / 2 + 4 * j, 4 * j};
}

// Heads [h0, h1) of a token, a head's row by 2^lane_bits lanes, two rows of a group in flight.
// kTurned: queries or keys, normed by `weight` (NULL: not) and turned; else values, copied.  All
// lanes of a warp call with the same range.
template <typename Src, typename Dst, bool kInterleaved, bool kTurned>
__device__ __forceinline__ void rotate_heads(const RotateParams& p, const Src* from, int64_t src_head,
                                             Dst* to, int64_t dst_head, int h0, int h1,
                                             const float* weight, const Place& at, bool write,
                                             bool read, const float (&c)[4], const float (&s)[4]) {
  using In = Quad<Src>;
  using Out = Quad<Dst>;
  constexpr int kAhead = 2;
  const int lanes = 1 << p.lane_bits, groups = kRotLanes >> p.lane_bits;
  const int group = (int)(threadIdx.x % kRotLanes) >> p.lane_bits;
  float4 wa, wb;
  if (kTurned && weight) {  // aligned to 4 bytes only
    wa = make_float4(weight[at.a], weight[at.a + 1], weight[at.a + 2], weight[at.a + 3]);
    wb = make_float4(weight[at.b], weight[at.b + 1], weight[at.b + 2], weight[at.b + 3]);
  }
  for (int first = h0; first < h1; first += kAhead * groups) {
    typename In::Load x[kAhead][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = first + u * groups + group;
      x[u][0] = x[u][1] = typename In::Load{};
      if (read && h < h1 && DSPARK_CHECK(at.a + 4 <= p.dim && at.b + 4 <= p.dim)) {
        x[u][0] = __ldcs(reinterpret_cast<const typename In::Load*>(from + h * src_head + at.a));
        x[u][1] = __ldcs(reinterpret_cast<const typename In::Load*>(from + h * src_head + at.b));
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      // no row of the token is left (for all lanes).  32 heads of 64 in f16, 384 tokens 5.2 us without
      // it, 4.6 with it; 16,384 tokens in fp32 98.9 and 101.2.
      if (sizeof(Src) == 2 && u > 0 && first + u * groups >= h1) break;
      const int h = first + u * groups + group;
      float4 a = In::widen(x[u][0]), b = In::widen(x[u][1]);
      if constexpr (kTurned) {
        if (weight) {
          float sum = a.x * a.x + a.y * a.y + a.z * a.z + a.w * a.w;
          sum += b.x * b.x + b.y * b.y + b.z * b.z + b.w * b.w;
          for (int m = lanes >> 1; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
          const float f = rsqrtf(sum / (float)p.dim + p.eps);
          a = scale4(a, f, wa);
          b = scale4(b, f, wb);
        }
        if (at.pair >= 0) turn8<kInterleaved>(a, b, c, s);
      }
      if (!write || h >= h1 || !DSPARK_CHECK(at.a + 4 <= p.dim && at.b + 4 <= p.dim)) continue;
      if (!read) a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // padding
      *reinterpret_cast<typename Out::Load*>(to + h * dst_head + at.a) = Out::round(a);
      *reinterpret_cast<typename Out::Load*>(to + h * dst_head + at.b) = Out::round(b);
    }
  }
}

// Bound by HBM: every element is read once and written once, the turns of a token computed once for
// all its heads.  Few registers, so that four CTAs of an SM hide one another's starts: 16,384
// tokens of 48 rows of 128, fp32 to bf16, take 98 us (6.2 TB/s; with five CTAs 100, and with all of
// a token's rows in one loop, 106 registers and two CTAs 141), in bf16 87 us (with three, four, five,
// six CTAs 98, 87, 85, 86; 2,400 tokens 17.7, 13.6, 15.2, 16.9).  Two rows in flight: one alone takes
// 100 us in bf16, four 95.
template <typename Src, typename Dst, bool kInterleaved>
__global__ void __launch_bounds__(kRotThreads, 4)
    rotate_kernel(const RotateParams p) {
  __shared__ float2 turns[kRotTokens][kMaxRot / 2];
  const int sub = threadIdx.x / kRotLanes, t = threadIdx.x % kRotLanes;
  const int64_t token = (int64_t)blockIdx.x * kRotTokens + sub;
  const bool mine = token < p.n_tokens;
  const int position = mine ? p.positions[token] : -1;
  const bool live = position >= 0;
  for (int i = t; i < p.rot_dim / 2; i += kRotLanes) {
    const uint64_t entry = __ldg(p.table + i);  // beside the position's load
    if (live && DSPARK_CHECK(i < kMaxRot / 2)) turns[sub][i] = turn_of(position, entry, p.magnitude);
  }

  const int lane = t & ((1 << p.lane_bits) - 1);
  const bool inside = lane < p.dim / 8;
  const Place at = place_of<kInterleaved>(inside ? lane : 0, p.rot_start, p.rot_dim);

  // the token's source, and the place of its keys and values
  const int64_t src = p.src_rows && mine ? p.src_rows[token] : token;
  bool store = mine && src >= 0 && src < p.n_src;
  int64_t to = token * p.ko_token;
  if (p.slots) {
    const int slot = mine ? p.slots[token] : -1;
    store = store && live && slot >= 0 && slot < p.n_blocks * p.page;
    const int block = store ? slot / p.page : 0;
    to = block * p.block_stride + (int64_t)(slot - block * p.page) * p.ko_token;
  }
  if (!store) to = 0;
  store = store && inside;

  __syncthreads();
  float c[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 turn = at.pair >= 0 && live ? turns[sub][at.pair + i] : make_float2(1.0f, 0.0f);
    c[i] = turn.x;
    s[i] = turn.y;
  }
  // this CTA's rows of a token: queries, keys and values one after the other
  const int begin = blockIdx.y * p.per, end = min(p.rows, begin + p.per), keys = p.heads + p.kv_heads;
  if (begin < p.heads)
    rotate_heads<Src, Dst, kInterleaved, true>(
        p, static_cast<const Src*>(p.q) + (mine ? token * p.q_token : 0), p.q_head,
        static_cast<Dst*>(p.q_out) + (mine ? token * p.qo_token : 0), p.qo_head, begin,
        min(end, p.heads), p.q_weight, at, mine && inside, live && inside, c, s);
  const int64_t from = store ? src * p.k_token : 0;
  if (begin < keys && end > p.heads)
    rotate_heads<Src, Dst, kInterleaved, true>(
        p, static_cast<const Src*>(p.k) + from, p.k_head, static_cast<Dst*>(p.k_out) + to, p.ko_head,
        max(begin - p.heads, 0), min(end - p.heads, p.kv_heads), p.k_weight, at, store,
        store && live, c, s);
  if (end > keys)
    rotate_heads<Src, Dst, kInterleaved, false>(
        p, static_cast<const Src*>(p.v) + from, p.k_head, static_cast<Dst*>(p.v_out) + to, p.ko_head,
        max(begin - keys, 0), end - keys, nullptr, at, store, store, c, s);
}

// -------------------------------------------------- rows of a latent cache
constexpr int kLatentThreads = 256;
constexpr int kMaxLatent = 512;

struct LatentWriteParams {
  const void* c;
  const void* r;
  int64_t c_token, r_token;
  int n_src, n_tokens, latent, rope;
  const float* weight;
  float eps;
  const int32_t* positions;
  const uint64_t* table;
  float magnitude;
  void* cache;
  int64_t block_stride, token_stride;
  int n_blocks, page;
  const int32_t* slots;
  const int32_t* src_rows;
};

// A warp per token: its latent vector in one go for the norm, and the rotated
// part by its first lanes, with one turn computed by each lane.  Bound by HBM.
template <typename Src, typename Dst, bool kInterleaved>
__global__ void __launch_bounds__(kLatentThreads) latent_write_kernel(const LatentWriteParams p) {
  using In = Quad<Src>;
  using Out = Quad<Dst>;
  constexpr int kPer = kMaxLatent / 128;  // fours of a lane
  const int lane = threadIdx.x & 31;
  const int64_t token = ((int64_t)blockIdx.x * kLatentThreads + threadIdx.x) >> 5;
  if (token >= p.n_tokens) return;  // a whole warp, as in what follows
  const int slot = p.slots[token], position = p.positions[token];
  const int64_t src = p.src_rows ? p.src_rows[token] : token;
  if (slot < 0 || slot >= p.n_blocks * p.page || position < 0 || src < 0 || src >= p.n_src) return;
  const Src* c = static_cast<const Src*>(p.c) + src * p.c_token;
  const Src* r = static_cast<const Src*>(p.r) + src * p.r_token;
  const int block = slot / p.page;
  Dst* to = static_cast<Dst*>(p.cache) + block * p.block_stride +
            (int64_t)(slot - block * p.page) * p.token_stride;
  typename In::Load x[kPer], ra{}, rb{};
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int d = (i * 32 + lane) * 4;
    x[i] = typename In::Load{};
    if (d < p.latent && DSPARK_CHECK(d + 4 <= p.latent))
      x[i] = __ldcs(reinterpret_cast<const typename In::Load*>(c + d));
  }
  const bool turning = lane < p.rope / 8;
  const Place at = place_of<kInterleaved>(turning ? lane : 0, 0, p.rope);
  if (turning && DSPARK_CHECK(at.b + 4 <= p.rope)) {
    ra = __ldcs(reinterpret_cast<const typename In::Load*>(r + at.a));
    rb = __ldcs(reinterpret_cast<const typename In::Load*>(r + at.b));
  }
  float2 turn = make_float2(1.0f, 0.0f);
  if (lane < p.rope / 2) turn = turn_of(position, p.table[lane], p.magnitude);
  float cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs[i] = __shfl_sync(0xffffffffu, turn.x, (4 * lane + i) & 31);
    sn[i] = __shfl_sync(0xffffffffu, turn.y, (4 * lane + i) & 31);
  }
  float f = 1.0f;
  const bool whole = reinterpret_cast<uintptr_t>(p.weight) % 16 == 0;  // the weights' fours
  if (p.weight) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float4 v = In::widen(x[i]);
      sum += v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
    }
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    f = rsqrtf(sum / (float)p.latent + p.eps);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int d = (i * 32 + lane) * 4;
    if (d >= p.latent) continue;
    float4 v = In::widen(x[i]);
    if (p.weight) {
      const float* w = p.weight + d;
      v = scale4(v, f, whole ? *reinterpret_cast<const float4*>(w)
                             : make_float4(w[0], w[1], w[2], w[3]));
    }
    *reinterpret_cast<typename Out::Load*>(to + d) = Out::round(v);
  }
  if (turning) {
    float4 a = In::widen(ra), b = In::widen(rb);
    turn8<kInterleaved>(a, b, cs, sn);
    *reinterpret_cast<typename Out::Load*>(to + p.latent + at.a) = Out::round(a);
    *reinterpret_cast<typename Out::Load*>(to + p.latent + at.b) = Out::round(b);
  }
}

template <template <typename, typename, bool> class Launch, typename... Args>
cudaError_t by_types(int src, int dst, bool interleaved, const Args&... args) {
  using B = __nv_bfloat16;
  using H = __half;
#define DSPARK_PICK(S, D)                                  \
  return interleaved ? Launch<S, D, true>::launch(args...) \
                     : Launch<S, D, false>::launch(args...)
  if (src == DSPARK_F32 && dst == DSPARK_F32) DSPARK_PICK(float, float);
  if (src == DSPARK_F32 && dst == DSPARK_BF16) DSPARK_PICK(float, B);
  if (src == DSPARK_F32) DSPARK_PICK(float, H);
  if (src == DSPARK_BF16) DSPARK_PICK(B, B);
  DSPARK_PICK(H, H);
#undef DSPARK_PICK
}

template <typename Src, typename Dst, bool kInterleaved>
struct LaunchRotate {
  static cudaError_t launch(const RotateParams& p, dim3 grid, cudaStream_t stream) {
    rotate_kernel<Src, Dst, kInterleaved><<<grid, kRotThreads, 0, stream>>>(p);
    return cudaGetLastError();
  }
};
template <typename Src, typename Dst, bool kInterleaved>
struct LaunchLatentWrite {
  static cudaError_t launch(const LatentWriteParams& p, unsigned grid, cudaStream_t stream) {
    if constexpr (!std::is_same_v<Dst, float>) {
      latent_write_kernel<Src, Dst, kInterleaved><<<grid, kLatentThreads, 0, stream>>>(p);
      return cudaGetLastError();
    } else {
      return cudaErrorInvalidValue;  // no cache of 32 bits
    }
  }
};

}  // namespace

cudaError_t launch_rotate(const void* q, const void* k, const void* v, int src_dtype,
                          int64_t q_token, int64_t q_head, int64_t k_token, int64_t k_head,
                          int n_src, int n_tokens, int heads, int kv_heads, int dim,
                          const float* q_weight, const float* k_weight, float eps,
                          const int32_t* positions, const uint64_t* table, int rot_start,
                          int rot_dim, bool interleaved, float magnitude, void* q_out,
                          int64_t qo_token, int64_t qo_head, void* k_out, void* v_out,
                          int dst_dtype, int64_t block_stride, int64_t ko_token, int64_t ko_head,
                          int n_blocks, int page, const int32_t* slots, const int32_t* src_rows,
                          cudaStream_t stream) {
  RotateParams p;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_token = q_token;
  p.q_head = q_head;
  p.k_token = k_token;
  p.k_head = k_head;
  p.n_src = n_src;
  p.n_tokens = n_tokens;
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.rows = heads + (v ? 2 : 1) * kv_heads;
  p.dim = dim;
  p.lane_bits = 0;
  while ((8 << p.lane_bits) < dim) ++p.lane_bits;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.eps = eps;
  p.positions = positions;
  p.table = table;
  p.rot_start = rot_start;
  p.rot_dim = rot_dim;
  p.magnitude = magnitude;
  p.q_out = q_out;
  p.qo_token = qo_token;
  p.qo_head = qo_head;
  p.k_out = k_out;
  p.v_out = v_out;
  p.ko_token = ko_token;
  p.ko_head = ko_head;
  p.block_stride = block_stride;
  p.n_blocks = n_blocks;
  p.page = page;
  p.slots = slots;
  p.src_rows = src_rows;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((int64_t)n_tokens + kRotTokens - 1) / kRotTokens;
  const int groups = kRotLanes >> p.lane_bits;
  // Few tokens: a token's rows go to several CTAs, until there are two an SM; more of them compute
  // the turns too often.  32 + 8 + 8 heads of 128, bf16, on 152 SMs until 1, 152, 304, 456, 608 CTAs:
  // 1 token 6.4, 2.5, 2.5, 2.5, 2.5 us; 384 tokens 7.0, 5.4, 5.0, 5.0, 4.8; 768: 8.1, 8.1, 6.4, 6.2,
  // 7.5; 2,400: 12.7, 12.7, 12.6, 12.7, 14.1.
  const int most = (p.rows + groups - 1) / groups;
  const int64_t wanted = (2 * (int64_t)sms + tiles - 1) / tiles;
  const int splits = wanted < most ? (int)wanted : most;
  p.per = (p.rows + splits - 1) / splits;
  // whole groups: 28 + 4 + 4 heads of 64, 384 tokens 4.6 -> 3.8 us
  if (splits > 1) p.per = (p.per + groups - 1) / groups * groups;
  const dim3 grid((unsigned)tiles, (unsigned)((p.rows + p.per - 1) / p.per));
  return by_types<LaunchRotate>(src_dtype, dst_dtype, interleaved, p, grid, stream);
}

cudaError_t launch_latent_write(const void* c, int64_t c_token, const void* r, int64_t r_token,
                                int src_dtype, int n_src, int latent, int rope,
                                const float* weight, float eps, const int32_t* positions,
                                const uint64_t* table, bool interleaved, float magnitude,
                                void* cache, int cache_dtype, int64_t block_stride,
                                int64_t token_stride, int n_blocks, int page,
                                const int32_t* slots, const int32_t* src_rows, int n_tokens,
                                cudaStream_t stream) {
  LatentWriteParams p;
  p.c = c;
  p.r = r;
  p.c_token = c_token;
  p.r_token = r_token;
  p.n_src = n_src;
  p.n_tokens = n_tokens;
  p.latent = latent;
  p.rope = rope;
  p.weight = weight;
  p.eps = eps;
  p.positions = positions;
  p.table = table;
  p.magnitude = magnitude;
  p.cache = cache;
  p.block_stride = block_stride;
  p.token_stride = token_stride;
  p.n_blocks = n_blocks;
  p.page = page;
  p.slots = slots;
  p.src_rows = src_rows;
  const int64_t threads = (int64_t)n_tokens * 32;
  const unsigned grid = (unsigned)((threads + kLatentThreads - 1) / kLatentThreads);
  return by_types<LaunchLatentWrite>(src_dtype, cache_dtype, interleaved, p, grid, stream);
}

DSPARK_CHECK_COLLECTOR(rotate)

}  // namespace dspark
