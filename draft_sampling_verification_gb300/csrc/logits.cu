// logits.cu -- dspark_logits_process: penalties for repeated tokens, biases
// and grammar masks on logit rows.
//
// A row is read and written once (2 V e bytes); the penalties and biases
// touch only the tokens of the request's text, drafts and bias list, a few
// thousand of V.  So the row goes through as a masked copy, and the touched
// tokens are then computed again from the input, each once, from a list with
// its count.  A CTA takes one slice of the vocabulary of one request: it
// scans the text once, counts the slice's tokens in shared memory (integer
// atomics: the counts do not depend on their order) and uses list and counts
// for its share of the request's rows.
#include <cuda_bf16.h>

#define DSPARK_TU 11  // this file's number in the checked build's site codes
#include "common.cuh"

namespace dspark {

namespace {

constexpr int kLThreads = 256;
constexpr uint32_t kCountBits = 0x00FFFFFFu;  // occurrences in the generated text
constexpr uint32_t kListed = 1u << 31;        // on the list of touched tokens
constexpr uint32_t kPrompt = 1u << 30;        // occurs in the prompt
constexpr uint32_t kDrafted = 1u << 29;       // equals one of the drafts

struct LParams {
  const void* x;
  int64_t ld;
  int B, rows, V;
  const int32_t* history;
  int64_t history_ld;
  const int32_t* prompt_len;
  const int32_t* history_len;
  const int32_t* drafts;
  int n_drafts;
  const uint64_t* row_mask;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* bias_ids;
  const float* bias_values;
  int max_bias;
  const int32_t* n_bias;
  const uint32_t* words;
  int64_t mask_ld;
  int n_masks;
  const int32_t* mask_rows;
  void* out;
  int64_t ld_out;
  int32_t* status;
  int slice;       // vocabulary ids per CTA (a multiple of 256)
  int row_step;    // rows per CTA
  int bias_cap;    // entries of the shared bias array
};

template <typename T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float widen<uint16_t>(uint16_t v) {
  return bf16_to_f32(v);
}
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ uint16_t narrow<uint16_t>(float v) {
  const __nv_bfloat16 h = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&h);
}

// the mask bits of tokens v .. v+n-1 (n <= 32) of a row's mask, from bit 0
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* words, int v, int n, int n_words) {
  const int w = v >> 5, s = v & 31;
  const uint32_t lo = __ldg(words + w);
  const uint32_t hi = (s + n > 32 && w + 1 < n_words) ? __ldg(words + w + 1) : 0u;
  return __funnelshift_r(lo, hi, s);
}

template <typename T>
__device__ __forceinline__ T minus_inf() {
  return narrow<T>(-INFINITY);
}

// A row's part in the CTA's slice, for the copy.
template <typename T>
struct RowPart {
  const T* x;             // element 0 is token v0
  T* out;
  const uint32_t* words;  // the row's mask, or NULL
  int head, vecs;         // 16-byte pieces [head, head + vecs * kVec); the rest one by one
  bool copied;            // false: in place and without a mask, nothing to do
};

// Copies the slice's n elements of `rows` rows, with -infinity where a row's
// mask has a 0.  Sixteen bytes at a time where a row's source and destination
// share their alignment, else one element at a time.  The pieces of all rows
// stand in one line, so that every thread has kUnroll loads in flight
// whatever the rows' and the slice's sizes.
template <typename T>
__device__ __forceinline__ void masked_copy(const RowPart<T>* parts, int rows, int slice, int v0,
                                            int n, int n_words) {
  constexpr int kVec = 16 / sizeof(T);
  constexpr int kUnroll = 6;
  const int per = slice / kVec;  // places of a row in the line
  const int all = rows * per;
  for (int i0 = threadIdx.x; i0 < all; i0 += kUnroll * kLThreads) {
    uint4 q[kUnroll];
    uint32_t bits[kUnroll];
    T* to[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kLThreads;
      const int r = i / per, at = i - r * per;
      to[u] = nullptr;
      if (i >= all) continue;
      const RowPart<T> part = parts[r];
      if (at >= part.vecs) continue;
      const int e = part.head + at * kVec;
      q[u] = __ldcs(reinterpret_cast<const uint4*>(part.x + e));
      bits[u] = part.words ? mask_bits(part.words, v0 + e, kVec, n_words) : ~0u;
      to[u] = part.out + e;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!to[u]) continue;
      T* e = reinterpret_cast<T*>(&q[u]);
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (!((bits[u] >> j) & 1u)) e[j] = minus_inf<T>();
      __stcs(reinterpret_cast<uint4*>(to[u]), q[u]);
    }
  }
  for (int r = 0; r < rows; ++r) {
    const RowPart<T> part = parts[r];
    if (!part.copied) continue;
    const int tail = part.head + part.vecs * kVec;
    for (int i = threadIdx.x; i < part.head + (n - tail); i += kLThreads) {
      const int e = i < part.head ? i : tail + (i - part.head);
      const bool on = !part.words || (mask_bits(part.words, v0 + e, 1, n_words) & 1u);
      part.out[e] = on ? part.x[e] : minus_inf<T>();
    }
  }
}

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kLThreads) logits_process_kernel(const LParams p) {
  extern __shared__ uint32_t smem[];
  uint32_t* table = smem;                                         // [slice]
  float* bias = reinterpret_cast<float*>(table + p.slice);        // [bias_cap], by list place
  uint16_t* list = reinterpret_cast<uint16_t*>(bias + p.bias_cap);  // [slice] touched tokens
  __shared__ int32_t s_draft[DSPARK_MAX_NODES];
  __shared__ uint32_t s_count, s_twice;
  __shared__ RowPart<T> s_part[DSPARK_MAX_NODES];
  __shared__ uint64_t s_seen[DSPARK_MAX_NODES];  // the drafts before each row
  const int tid = threadIdx.x;
  const int b = blockIdx.y;
  const int v0 = blockIdx.x * p.slice;
  const int n = min(p.slice, p.V - v0);
  const int n_words = (p.V + 31) >> 5;
  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out);

  const float R = p.repetition ? p.repetition[b] : 1.0f;
  const float F = p.frequency ? p.frequency[b] : 0.0f;
  const float P = p.presence ? p.presence[b] : 0.0f;
  const bool bad = !(R > 0.0f && R < INFINITY) || !(fabsf(F) < INFINITY) || !(fabsf(P) < INFINITY);
  if (tid == 0 && blockIdx.x == 0 && blockIdx.z == 0)
    p.status[b] = bad ? DSPARK_ST_BAD_PENALTY : DSPARK_ST_OK;
  if (bad) {
    for (int r = blockIdx.z * p.row_step; r < min(p.rows, (int)(blockIdx.z + 1) * p.row_step);
         ++r) {
      T* row = out + ((int64_t)b * p.rows + r) * p.ld_out + v0;
      for (int i = tid; i < n; i += kLThreads) row[i] = minus_inf<T>();
    }
    return;
  }

  // this CTA's rows: r0, r0 + 1, ...
  const int r0 = blockIdx.z * p.row_step, rows = min(p.row_step, p.rows - r0);
  if (tid < rows) {
    constexpr int kVec = 16 / sizeof(T);
    const int64_t row = (int64_t)b * p.rows + r0 + tid;
    RowPart<T> part;
    part.x = x + row * p.ld + v0;
    part.out = out + row * p.ld_out + v0;
    part.words = nullptr;
    if (p.words) {
      const int64_t m = p.mask_rows ? (int64_t)p.mask_rows[row] : row;
      if (m >= 0 && m < p.n_masks) part.words = p.words + m * p.mask_ld;
    }
    part.copied = part.words || (const void*)part.x != (const void*)part.out;
    const uintptr_t ax = reinterpret_cast<uintptr_t>(part.x) & 15;
    part.head = n;
    part.vecs = 0;
    if (!part.copied) {
      part.head = 0;
    } else if (ax == (reinterpret_cast<uintptr_t>(part.out) & 15)) {
      part.head = min(n, (int)(((16 - ax) & 15) / sizeof(T)));
      part.vecs = (n - part.head) / kVec;
    }
    s_part[tid] = part;
    s_seen[tid] = p.row_mask ? p.row_mask[row] : (1ull << (r0 + tid)) - 1ull;
  }
  __syncthreads();
  // the rows go through first: the copies are in flight while the text is
  // counted.  In place, a row without a mask is left as it is; a token that
  // its mask lets through still holds its input below.
  masked_copy(s_part, rows, p.slice, v0, n, n_words);

  for (int i = tid; i < n; i += kLThreads) table[i] = 0u;
  if (tid == 0) s_count = s_twice = 0u;
  if (tid < p.n_drafts) s_draft[tid] = p.drafts[(int64_t)b * p.n_drafts + tid];
  __syncthreads();

  // the slice's biases: the first entry of an id owns it and adds up the
  // later ones in list order; owners come first on the list of touched tokens
  int n_bias = 0;
  if (p.max_bias > 0) n_bias = max(0, min(p.max_bias, p.n_bias ? p.n_bias[b] : p.max_bias));
  if (n_bias > 0) {
    const int32_t* ids = p.bias_ids + (int64_t)b * p.max_bias;
    const float* values = p.bias_values + (int64_t)b * p.max_bias;
    for (int i = tid; i < n_bias; i += kLThreads) {
      const uint32_t t = (uint32_t)(ids[i] - v0);
      if (t < (uint32_t)n && atomicMax(&table[t], 65536u - (uint32_t)i) != 0u) s_twice = 1u;
    }
    __syncthreads();
    const bool twice = s_twice != 0u;
    for (int i = tid; i < n_bias; i += kLThreads) {
      const uint32_t t = (uint32_t)(ids[i] - v0);
      if (t >= (uint32_t)n || table[t] != 65536u - (uint32_t)i) continue;
      float sum = values[i];
      if (twice)
        for (int k = i + 1; k < n_bias; ++k)
          if (ids[k] == ids[i]) sum = __fadd_rn(sum, values[k]);
      const uint32_t at = atomicAdd(&s_count, 1u);
      if (DSPARK_CHECK(at < (uint32_t)p.bias_cap)) {
        list[at] = (uint16_t)t;
        bias[at] = sum;
      }
    }
    __syncthreads();
    for (int i = tid; i < (int)s_count; i += kLThreads) table[list[i]] = kListed;
    __syncthreads();
  }
  const int n_biased = (int)s_count;
  __syncthreads();

  // the text
  if (p.history) {
    const int len = (int)max((int64_t)0, min(p.history_ld, (int64_t)p.history_len[b]));
    const int prompt = p.prompt_len ? max(0, min(len, p.prompt_len[b])) : 0;
    const int32_t* text = p.history + (int64_t)b * p.history_ld;
    for (int i = tid; i < len; i += kLThreads) {
      const uint32_t t = (uint32_t)(text[i] - v0);
      if (t >= (uint32_t)n) continue;
      const uint32_t old = i < prompt ? atomicOr(&table[t], kPrompt | kListed)
                                      : atomicAdd(&table[t], 1u);
      if (old & kListed) continue;
      // the one that sets the bit lists the token
      if (i < prompt || !(atomicOr(&table[t], kListed) & kListed)) {
        const uint32_t at = atomicAdd(&s_count, 1u);
        if (DSPARK_CHECK(at < (uint32_t)p.slice)) list[at] = (uint16_t)t;
      }
    }
  }
  if (tid < p.n_drafts) {
    const uint32_t t = (uint32_t)(s_draft[tid] - v0);
    if (t < (uint32_t)n && !(atomicOr(&table[t], kDrafted | kListed) & kListed)) {
      const uint32_t at = atomicAdd(&s_count, 1u);
      if (DSPARK_CHECK(at < (uint32_t)p.slice)) list[at] = (uint16_t)t;
    }
  }
  __syncthreads();
  const int touched = (int)s_count;

  // each touched token of each row, from its input
  for (int k = tid; k < touched * rows; k += kLThreads) {
    const int r = k / touched, i = k - r * touched;
    const RowPart<T> part = s_part[r];
    const int t = list[i];
    if (part.words && !(mask_bits(part.words, v0 + t, 1, n_words) & 1u)) continue;
    const uint32_t w = table[t];
    uint32_t c = w & kCountBits;
    if (w & kDrafted)
      for (int j = 0; j < p.n_drafts; ++j)
        if (((s_seen[r] >> j) & 1ull) && s_draft[j] == v0 + t) ++c;
    float y = widen(part.x[t]);
    if (c > 0u || (w & kPrompt)) y = y > 0.0f ? __fdiv_rn(y, R) : __fmul_rn(y, R);
    y = __fsub_rn(y, __fmul_rn(F, (float)c));
    if (c > 0u) y = __fsub_rn(y, P);
    if (i < n_biased) y = __fadd_rn(y, bias[i]);
    part.out[t] = narrow<T>(y);
  }
}

cudaError_t launch_logits_process(
    const void* x, int dtype, int64_t ld, int B, int rows, int V, const int32_t* history,
    int64_t history_ld, const int32_t* prompt_len, const int32_t* history_len,
    const int32_t* drafts, int n_drafts, const uint64_t* row_mask, const float* repetition,
    const float* frequency, const float* presence, const int32_t* bias_ids,
    const float* bias_values, int max_bias, const int32_t* n_bias, const uint32_t* words,
    int64_t mask_ld, int n_masks, const int32_t* mask_rows, void* out, int64_t ld_out,
    int32_t* status, cudaStream_t stream) {
  LParams p;
  p.x = x;
  p.ld = ld;
  p.B = B;
  p.rows = rows;
  p.V = V;
  p.history = history;
  p.history_ld = history_ld;
  p.prompt_len = prompt_len;
  p.history_len = history_len;
  p.drafts = drafts;
  p.n_drafts = n_drafts;
  p.row_mask = row_mask;
  p.repetition = repetition;
  p.frequency = frequency;
  p.presence = presence;
  p.bias_ids = bias_ids;
  p.bias_values = bias_values;
  p.max_bias = max_bias;
  p.n_bias = n_bias;
  p.words = words;
  p.mask_ld = mask_ld;
  p.n_masks = n_masks;
  p.mask_rows = mask_rows;
  p.out = out;
  p.ld_out = ld_out;
  p.status = status;
  p.slice = 4096;
  const int slices = (V + p.slice - 1) / p.slice;
  // a CTA takes all rows of its request, as the text is counted once for
  // them, unless that leaves SMs without work
  const int64_t ctas = (int64_t)slices * B, wanted = 1024;
  const int parts = (int)(ctas >= wanted ? 1 : (wanted + ctas - 1) / ctas);
  p.row_step = parts >= rows ? 1 : (rows + parts - 1) / parts;
  p.bias_cap = max_bias < p.slice ? max_bias : p.slice;
  const size_t smem = (size_t)p.slice * 6 + (size_t)p.bias_cap * 4;
  const dim3 grid(slices, B, (rows + p.row_step - 1) / p.row_step);
  if (dtype == DSPARK_F32)
    logits_process_kernel<float><<<grid, kLThreads, smem, stream>>>(p);
  else
    logits_process_kernel<uint16_t><<<grid, kLThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

DSPARK_CHECK_COLLECTOR(logits)

}  // namespace dspark
