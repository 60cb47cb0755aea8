// logits.cu -- dspark_logits_process: penalties for repeated tokens, biases
// and grammar masks on logit rows.
//
// A row is read and written once (2 V e bytes); the penalties and biases
// touch only the tokens of the request's text, drafts and bias list, a few
// thousand of V.  So the rows go through as masked copies, and the touched
// tokens are then computed again from the input, each once.  A CTA takes one
// slice of the vocabulary of one request: it scans the text once, counts the
// slice's tokens in shared memory (integer atomics: the counts do not depend
// on their order), lists the touched ones, and goes with list and counts over
// its share of the request's rows; tokens with more than one bias, which are
// added in list order, in a pass of their own.  Bound by HBM; slices are long, since each
// scans the whole text and has its own start and end.  256 requests of six
// bf16 rows of 129,280 under masks take 135 us (5.9 TB/s), 64 of fp32 rows 72
// us (5.5 TB/s), one request of six rows 5 us.
#include <cuda_bf16.h>

#include <type_traits>

#define DSPARK_TU 11  // this file's number in the checked build's site codes
#include "common.cuh"

namespace dspark {

namespace {

constexpr int kCopyThreads = 512, kTextThreads = 128;
constexpr int kLThreads = kCopyThreads + kTextThreads;
constexpr int kSliceBytes = 32768, kMinSliceBytes = 4096;  // of a row, per CTA
constexpr size_t kMaxSmem = kSliceBytes / 2 * 10;          // counts, biases and list
constexpr uint32_t kCountBits = 0x00FFFFFFu;  // occurrences in the generated text
constexpr uint32_t kListed = 1u << 31;        // on the list of touched tokens
constexpr uint32_t kPrompt = 1u << 30;        // occurs in the prompt
constexpr uint32_t kDrafted = 1u << 29;       // equals one of the drafts
constexpr uint32_t kRepeated = 1u << 28;      // more than one bias
constexpr uint32_t kOwner = 0x1FFFFu;         // 65536 - list place of a token's first bias

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
  int slice;       // vocabulary ids per CTA (a power of two)
  int row_step;    // rows per CTA
  int bias_cap;    // entries of the shared bias array, and of the list: the most
  int list_cap;    // tokens of a slice that can be touched
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

// the mask bits of elements e .. e + 31 of a slice with n_words words, from bit 0
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* words, int e, int n_words) {
  const int w = e >> 5;
  return __funnelshift_r(__ldg(words + w), __ldg(words + min(w + 1, n_words - 1)), e & 31);
}

template <typename T>
__device__ __forceinline__ T minus_inf() {
  return narrow<T>(-INFINITY);
}

// two bf16 logits with -infinity where the lower two of `bits` have a 0
__device__ __forceinline__ uint32_t masked_pair(uint32_t w, uint32_t bits) {
  const uint32_t keep = ((bits & 1u) | ((bits & 2u) << 15)) * 0xFFFFu;
  return (w & keep) | (0xFF80FF80u & ~keep);
}

// A row's part in the CTA's slice: n elements, of which element 0 is token v0.
template <typename T>
struct RowPart {
  const T* x;
  T* out;
  const uint32_t* words;  // the mask's words from the slice's first on, or NULL
  uint64_t seen;          // the drafts before the row
  int head, vecs;         // [head, head + vecs * kVec): 16-byte pieces of both sides
  bool copied;            // false: in place and without a mask
};

// A row's part to its place, with -infinity where its mask has a 0: sixteen
// bytes at a time where source and destination share their alignment, else
// one element at a time.  A slice has at most kUnroll pieces a thread, which
// are read without a branch (past the end: the last one again), so that all
// are in flight together.
template <typename T, bool kMasked>
__device__ __forceinline__ void copy_row(const RowPart<T>& part, int n, int n_words) {
  constexpr int kVec = 16 / sizeof(T);
  constexpr int kUnroll = kSliceBytes / 16 / kCopyThreads;
  const int head = part.head, vecs = part.vecs;
  const T* x = part.x;
  T* out = part.out;
  const uint32_t* words = part.words;
  const uint4* from = reinterpret_cast<const uint4*>(x + head);
  uint4* to = reinterpret_cast<uint4*>(out + head);
  if (vecs > 0) {
    uint4 q[kUnroll];
    uint32_t m[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int j = min((int)threadIdx.x + u * kCopyThreads, vecs - 1), e = head + j * kVec;
      q[u] = from[j];
      // a piece's bits lie in one word unless the row begins inside a piece
      if (kMasked)
        m[u] = head ? mask_bits(words, e, n_words) : __ldg(words + (e >> 5)) >> (e & 31);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int j = (int)threadIdx.x + u * kCopyThreads;
      if (j >= vecs) break;
      uint4 w = q[u];
      if constexpr (kMasked && sizeof(T) == 2) {
        w = make_uint4(masked_pair(w.x, m[u]), masked_pair(w.y, m[u] >> 2),
                       masked_pair(w.z, m[u] >> 4), masked_pair(w.w, m[u] >> 6));
      } else if constexpr (kMasked) {
        constexpr uint32_t kInf = 0xFF800000u;
        w = make_uint4(m[u] & 1u ? w.x : kInf, m[u] & 2u ? w.y : kInf, m[u] & 4u ? w.z : kInf,
                       m[u] & 8u ? w.w : kInf);
      }
      __stcs(to + j, w);
    }
  }
  const int tail = head + vecs * kVec;
  for (int i = threadIdx.x; i < head + n - tail; i += kCopyThreads) {
    const int e = i < head ? i : tail + (i - head);
    out[e] = !kMasked || (mask_bits(words, e, n_words) & 1u) ? x[e] : minus_inf<T>();
  }
}

// a barrier of the threads that count the text
__device__ __forceinline__ void text_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kTextThreads) : "memory");
}

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kLThreads, 2) logits_process_kernel(const LParams p) {
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t* table = smem;                                            // [slice]
  float* bias = reinterpret_cast<float*>(table + p.slice);           // [bias_cap], by list place
  uint16_t* list = reinterpret_cast<uint16_t*>(bias + p.bias_cap);   // [list_cap] touched tokens
  __shared__ int32_t s_draft[DSPARK_MAX_NODES];
  __shared__ uint32_t s_count, s_biased, s_repeated;
  __shared__ RowPart<T> s_part[DSPARK_MAX_NODES];
  const int tid = threadIdx.x;
  const int b = blockIdx.y;
  const int v0 = blockIdx.x * p.slice;
  const int n = min(p.slice, p.V - v0);
  const int n_words = (n + 31) >> 5;
  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out);
  // this CTA's rows: r0, r0 + 1, ...
  const int r0 = blockIdx.z * p.row_step, rows = min(p.row_step, p.rows - r0);

  const float R = p.repetition ? p.repetition[b] : 1.0f;
  const float F = p.frequency ? p.frequency[b] : 0.0f;
  const float P = p.presence ? p.presence[b] : 0.0f;
  const bool bad = !(R > 0.0f && R < INFINITY) || !(fabsf(F) < INFINITY) || !(fabsf(P) < INFINITY);
  if (tid == 0 && blockIdx.x == 0 && blockIdx.z == 0)
    p.status[b] = bad ? DSPARK_ST_BAD_PENALTY : DSPARK_ST_OK;
  if (bad) {
    for (int r = r0; r < r0 + rows; ++r) {
      T* row = out + ((int64_t)b * p.rows + r) * p.ld_out + v0;
      for (int i = tid; i < n; i += kLThreads) row[i] = minus_inf<T>();
    }
    return;
  }

  if (tid < rows) {
    const int64_t row = (int64_t)b * p.rows + r0 + tid;
    RowPart<T> part;
    part.x = x + row * p.ld + v0;
    part.out = out + row * p.ld_out + v0;
    part.words = nullptr;
    if (p.words) {
      const int64_t m = p.mask_rows ? (int64_t)p.mask_rows[row] : row;
      if (m >= 0 && m < p.n_masks) part.words = p.words + m * p.mask_ld + (v0 >> 5);
    }
    constexpr int kVec = 16 / sizeof(T);
    const uintptr_t ax = reinterpret_cast<uintptr_t>(part.x) & 15;
    part.copied = part.words || (const void*)part.x != (const void*)part.out;
    part.head = n;
    part.vecs = 0;
    if (part.copied && ax == (reinterpret_cast<uintptr_t>(part.out) & 15)) {
      part.head = min(n, (int)(((16 - ax) & 15) / sizeof(T)));
      part.vecs = (n - part.head) / kVec;
    }
    part.seen = p.row_mask ? p.row_mask[row] : (1ull << (r0 + tid)) - 1ull;
    s_part[tid] = part;
  }
  if (tid == 0) s_count = s_biased = s_repeated = 0u;
  __syncthreads();
  auto count_biases = [&]() -> int {
    return p.max_bias > 0 ? max(0, min(p.max_bias, p.n_bias ? p.n_bias[b] : p.max_bias)) : 0;
  };
  const int32_t* bias_ids = p.bias_ids + (int64_t)b * p.max_bias;
  const float* bias_values = p.bias_values + (int64_t)b * p.max_bias;
  // the slice's touched tokens: their counts, and the list of them
  auto count_text = [&](int t0) {
    for (int i = t0; i < p.slice / 4; i += kTextThreads)
      reinterpret_cast<uint4*>(table)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (t0 < p.n_drafts) s_draft[t0] = p.drafts[(int64_t)b * p.n_drafts + t0];
    text_sync();

    // the slice's biases: the first entry of an id owns it, later ones mark
    // it as repeated; owners come first on the list
    const int n_bias = count_biases();
    if (n_bias > 0) {
      for (int i = t0; i < n_bias; i += kTextThreads) {
        const uint32_t t = (uint32_t)(bias_ids[i] - v0);
        if (t < (uint32_t)n) atomicMax(&table[t], 65536u - (uint32_t)i);
      }
      text_sync();
      for (int i = t0; i < n_bias; i += kTextThreads) {
        const uint32_t t = (uint32_t)(bias_ids[i] - v0);
        if (t >= (uint32_t)n) continue;
        if ((*(volatile uint32_t*)&table[t] & kOwner) != 65536u - (uint32_t)i) {
          atomicOr(&table[t], kRepeated);
          s_repeated = 1u;
          continue;
        }
        const uint32_t at = atomicAdd(&s_count, 1u);
        if (DSPARK_CHECK(at < (uint32_t)p.bias_cap)) {
          list[at] = (uint16_t)t;
          bias[at] = bias_values[i];
        }
      }
      text_sync();
      if (t0 == 0) s_biased = s_count;
      for (int i = t0; i < (int)s_count; i += kTextThreads)
        table[list[i]] = kListed | (table[list[i]] & kRepeated);
      text_sync();
    }

    // the text
    if (p.history) {
      const int len = (int)max((int64_t)0, min(p.history_ld, (int64_t)p.history_len[b]));
      const int prompt = p.prompt_len ? max(0, min(len, p.prompt_len[b])) : 0;
      const int32_t* text = p.history + (int64_t)b * p.history_ld;
      constexpr int kAhead = 8;  // loads of a thread in flight
      for (int i0 = t0; i0 < len; i0 += kAhead * kTextThreads) {
        uint32_t at[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int i = i0 + u * kTextThreads;
          at[u] = i < len ? (uint32_t)(__ldg(text + i) - v0) : ~0u;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int i = i0 + u * kTextThreads;
          const uint32_t t = at[u];
          if (t >= (uint32_t)n) continue;
          const uint32_t old = i < prompt ? atomicOr(&table[t], kPrompt | kListed)
                                          : atomicAdd(&table[t], 1u);
          if (old & kListed) continue;
          // the one that sets the bit lists the token
          if (i < prompt || !(atomicOr(&table[t], kListed) & kListed)) {
            const uint32_t k = atomicAdd(&s_count, 1u);
            if (DSPARK_CHECK(k < (uint32_t)p.list_cap)) list[k] = (uint16_t)t;
          }
        }
      }
    }
    if (t0 < p.n_drafts) {
      const uint32_t t = (uint32_t)(s_draft[t0] - v0);
      if (t < (uint32_t)n && !(atomicOr(&table[t], kDrafted | kListed) & kListed)) {
        const uint32_t k = atomicAdd(&s_count, 1u);
        if (DSPARK_CHECK(k < (uint32_t)p.list_cap)) list[k] = (uint16_t)t;
      }
    }
  };

  // Most threads take the rows to their places while the others count.  In
  // place, a row without a mask is left as it is; a token that its mask lets
  // through still holds its input below.
  if (tid < kCopyThreads) {
    for (int r = 0; r < rows; ++r) {
      const RowPart<T>& part = s_part[r];
      if (part.words)
        copy_row<T, true>(part, n, n_words);
      else if (part.copied)
        copy_row<T, false>(part, n, n_words);
    }
  } else {
    count_text(tid - kCopyThreads);
  }
  __syncthreads();
  const int touched = (int)s_count, n_biased = (int)s_biased;

  // a touched token of a row, from its input; those with more than one bias apart, as the search
  // for the others in the list keeps the compiler from overlapping two tokens
  auto touch = [&](int k, auto repeated) {
    const int r = k / touched, i = k - r * touched;
    const RowPart<T>& part = s_part[r];
    const int t = list[i];
    if (part.words && !((__ldg(part.words + (t >> 5)) >> (t & 31)) & 1u)) return;
    const uint32_t w = table[t];
    if (decltype(repeated)::value != ((w & kRepeated) != 0u)) return;
    uint32_t c = w & kCountBits;
    if (w & kDrafted)
      for (int j = 0; j < p.n_drafts; ++j)
        if (((part.seen >> j) & 1ull) && s_draft[j] == v0 + t) ++c;
    float y = widen(part.x[t]);
    if (c > 0u || (w & kPrompt)) y = y > 0.0f ? __fdiv_rn(y, R) : __fmul_rn(y, R);
    y = __fsub_rn(y, __fmul_rn(F, (float)c));
    if (c > 0u) y = __fsub_rn(y, P);
    if (i < n_biased) y = __fadd_rn(y, bias[i]);
    if constexpr (decltype(repeated)::value) {  // its later biases, one addition each
      bool first = true;
      for (int e = 0, n_bias = count_biases(); e < n_bias; ++e) {
        if (bias_ids[e] != v0 + t) continue;
        if (!first) y = __fadd_rn(y, bias_values[e]);
        first = false;
      }
    }
    part.out[t] = narrow<T>(y);
  };
#pragma unroll 2
  for (int k = tid; k < touched * rows; k += kLThreads) touch(k, std::false_type());
  if (s_repeated)
    for (int k = tid; k < n_biased * rows; k += kLThreads)
      touch(k / n_biased * touched + k % n_biased, std::true_type());
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
  // Long slices where they make a CTA for every SM twice over (each scans the
  // whole text); else shorter ones, and where those do not a request's rows
  // shared out among CTAs.
  const int64_t wanted = 304;
  const int es = dtype == DSPARK_F32 ? 4 : 2;
  p.slice = kSliceBytes / es;
  auto ctas = [&] { return (int64_t)((V + p.slice - 1) / p.slice) * B; };
  while (p.slice > kMinSliceBytes / es && ctas() < wanted) p.slice /= 2;
  const int slices = (V + p.slice - 1) / p.slice;
  const int parts = (int)(ctas() >= wanted ? 1 : (wanted + ctas() - 1) / ctas());
  p.row_step = parts >= rows ? 1 : (rows + parts - 1) / parts;
  p.bias_cap = max_bias < p.slice ? max_bias : p.slice;
  const int64_t most = (history ? history_ld : 0) + n_drafts + max_bias;
  p.list_cap = most < p.slice ? (int)most : p.slice;
  const size_t smem = (size_t)p.slice * 4 + (size_t)p.bias_cap * 4 + (size_t)p.list_cap * 2;
  const dim3 grid(slices, B, (rows + p.row_step - 1) / p.row_step);
  auto launch = [&](auto* kernel) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kLThreads, smem, stream>>>(p);
    return cudaGetLastError();
  };
  return dtype == DSPARK_F32 ? launch(logits_process_kernel<float>)
                             : launch(logits_process_kernel<uint16_t>);
}

DSPARK_CHECK_COLLECTOR(logits)

}  // namespace dspark
