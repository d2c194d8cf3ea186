// Conditions on the target's logits of a round (include/dspark_logits.h):
// penalties for tokens that are there already, biases, a grammar's mask; and
// the token counts of the requests that the penalties go by.
//
// A row is read and written once, which is what bounds it.  A lane has 8
// neighbouring tokens; their counts, flags and biases of the request are loaded
// once and stay in registers over the request's rows, the row's own drafts are
// counted on the way.
//
// 2176 rows of 129280 bf16 logits with their masks: 232 us, 5.1 TB/s, what a
// copy of that size reaches.  32 rows of 151936: 12 us, of which the bytes are
// 6, the rest the launch and the chain of loads before the first store (its list
// of biases, the request's counts); new counts for their requests and 4000-token
// prompts 6 us, a round's tokens 2.5.
#include "cache.hpp"
#include "dspark_logits.h"

namespace dspark {

namespace {

constexpr int kT = 256;
constexpr int kEach = 8;                // tokens of a lane
constexpr int kSlice = kT * kEach;      // of a work group
constexpr int kMaxRows = kCacheMaxGamma + 1;
constexpr uint32_t kInPrompt = 0x8000u, kCount = 0x7FFFu;

// Rows of odd lengths begin anywhere: 16-byte accesses at the type's own
// alignment, which the memory system takes.
typedef u32x4 Words2 __attribute__((aligned(2)));
typedef f32x4 Words4 __attribute__((aligned(4)));

struct LogitsArgs {
  int R, gamma, V, nb;
  const void* in;
  const int32_t *row0, *ell, *x0, *x;
  const uint16_t* state;
  const float *repetition, *presence, *frequency;
  const int32_t* bias_tok;
  const float* bias;
  const uint8_t* mask;
  int64_t mask_row;  // bytes
  void* out;
  int rows_each;     // rows of a work group
};

// Eight words of 16 bits, n < 8 at a row's end.
__device__ __forceinline__ u32x4 load_words(const uint16_t* p, int n) {
  if (n == 8) return *reinterpret_cast<const Words2*>(p);
  u32x4 w{0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < n) w[e / 2] |= static_cast<uint32_t>(p[e]) << (16 * (e & 1));
  return w;
}
__device__ __forceinline__ void store_words(uint16_t* p, int n, u32x4 w) {
  if (n == 8) {
    *reinterpret_cast<Words2*>(p) = w;
    return;
  }
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < n) p[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
}

// Eight logits of a row, as stored and as numbers.
struct Logits16 {
  u32x4 w;
  __device__ __forceinline__ void load(const uint16_t* p, int n) { w = load_words(p, n); }
  __device__ __forceinline__ void get(float (&y)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
  }
  static __device__ __forceinline__ void store(uint16_t* p, int n, const float (&y)[8]) {
    store_words(p, n, u32x4{bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]), bf16_pair(y[4], y[5]), bf16_pair(y[6], y[7])});
  }
};
struct Logits32 {
  f32x4 w[2];
  __device__ __forceinline__ void load(const float* p, int n) {
    if (n == 8) {
      w[0] = reinterpret_cast<const Words4*>(p)[0];
      w[1] = reinterpret_cast<const Words4*>(p)[1];
      return;
    }
    w[0] = w[1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < n) w[e / 4][e % 4] = p[e];
  }
  __device__ __forceinline__ void get(float (&y)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = w[e / 4][e % 4];
  }
  static __device__ __forceinline__ void store(float* p, int n, const float (&y)[8]) {
    if (n == 8) {
      reinterpret_cast<Words4*>(p)[0] = f32x4{y[0], y[1], y[2], y[3]};
      reinterpret_cast<Words4*>(p)[1] = f32x4{y[4], y[5], y[6], y[7]};
      return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < n) p[e] = y[e];
  }
};

template <typename S, typename Logits>
__global__ __launch_bounds__(kT) void logits_kernel(LogitsArgs a) {
  __shared__ int lds_tok[kMaxRows];
  const int r = blockIdx.y;
  const int n_rows = rows_of(a.ell[r], a.gamma);
  const int i0 = blockIdx.z * a.rows_each, i1 = min(n_rows, i0 + a.rows_each);
  if (i0 >= i1) return;
  const int v0 = blockIdx.x * kSlice + threadIdx.x * kEach;
  const int n = max(0, min(kEach, a.V - v0));
  const int64_t row0 = a.row0 ? static_cast<int64_t>(a.row0[r]) : static_cast<int64_t>(r) * (a.gamma + 1);
  // a row's logits and mask are on their way while the row before is worked on
  auto load_row = [&](int i, Logits& y, uint32_t& allowed) {
    const int64_t row = row0 + i;
    if (n > 0) {
      y.load(static_cast<const S*>(a.in) + row * a.V + v0, n);
      allowed = a.mask ? a.mask[row * a.mask_row + (v0 >> 3)] : 0xFFu;
    }
  };
  Logits next{};
  uint32_t next_allowed = 0xFFu;
  load_row(i0, next, next_allowed);
  // the tokens that rows follow: the anchor, the drafts
  if (a.state)
    for (int j = threadIdx.x; j < i1; j += kT)
      lds_tok[j] = token_or_none(j == 0 ? a.x0[r] : a.x ? a.x[static_cast<int64_t>(r) * a.gamma + j - 1] : -1, a.V);
  int count[8];
  bool prompt[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) count[e] = 0, prompt[e] = false;
  if (a.state && n > 0) {
    const u32x4 w = load_words(a.state + static_cast<int64_t>(r) * a.V + v0, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t x = w[e / 2] >> (16 * (e & 1));
      count[e] = x & kCount;
      prompt[e] = (x & kInPrompt) != 0;
    }
  }
  const float rep = a.repetition ? a.repetition[r] : 1.f;
  const float pres = a.presence ? a.presence[r] : 0.f;
  const float freq = a.frequency ? a.frequency[r] : 0.f;
  // biases: 64 of the list at a time, those of this slice one by one
  float bias[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) bias[e] = 0.f;
  const int lane = threadIdx.x & 63, slice0 = blockIdx.x * kSlice;
  for (int j = 0; j < a.nb; j += 64) {
    const int64_t at = static_cast<int64_t>(r) * a.nb + j + lane;
    const int tok = j + lane < a.nb ? token_or_none(a.bias_tok[at], a.V) : -1;
    const float value = j + lane < a.nb ? a.bias[at] : 0.f;
    for (uint64_t here = __ballot(tok >= slice0 && tok < slice0 + kSlice); here; here &= here - 1) {
      const int l = __builtin_ctzll(here);
      const int t = __builtin_amdgcn_readlane(tok, l);
      const float b = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(value), l));
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (t == v0 + e) bias[e] += b;
    }
  }
  __syncthreads();
  if (a.state)
    for (int j = 0; j < i0; ++j) {
      const int t = lds_tok[j];
#pragma unroll
      for (int e = 0; e < 8; ++e) count[e] += t == v0 + e;
    }
  if (n == 0) return;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    const int64_t row = row0 + i;
    const Logits in = next;
    const uint32_t allowed = next_allowed;
    if (i + 1 < i1) load_row(i + 1, next, next_allowed);
    if (a.state) {
      const int t = lds_tok[i];
#pragma unroll
      for (int e = 0; e < 8; ++e) count[e] += t == v0 + e;
    }
    float y[8];
    in.get(y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (count[e] > 0 || prompt[e]) y[e] = y[e] > 0.f ? y[e] / rep : y[e] * rep;
      if (count[e] > 0) y[e] -= __builtin_fmaf(freq, static_cast<float>(count[e]), pres);
      y[e] += bias[e];
      if (!((allowed >> e) & 1u)) y[e] = neg_inf();
    }
    Logits::store(static_cast<S*>(a.out) + row * a.V + v0, n, y);
  }
}

// A slot's new history: a work group has a slice of the vocabulary, marks the
// prompt's tokens of it in LDS and writes every word of it.  Eight tokens of a
// thread are in flight (one at a time: 2.7 us more for the 32 prompts).  With
// slices of 65536 tokens those three calls take 24.6 us, of 16384 22.4, of 8192
// 21.8, of 4096 21.9; every slice reads the whole prompt.
constexpr int kPromptSlice = 8192;
__global__ __launch_bounds__(kT) void logits_prompt_kernel(int V, int64_t n, const int32_t* tokens,
                                                           const int32_t* start, const int32_t* count,
                                                           uint16_t* state) {
  __shared__ uint32_t seen[kPromptSlice / 32];
  const int r = blockIdx.y, v0 = blockIdx.x * kPromptSlice;
  const int m = count[r];
  if (m < 0) return;
  const int64_t first = max(static_cast<int64_t>(start[r]), static_cast<int64_t>(0));
  const int64_t last = min(static_cast<int64_t>(start[r]) + m, n);
  for (int i = threadIdx.x; i < kPromptSlice / 32; i += kT) seen[i] = 0;
  __syncthreads();
  constexpr int kAtOnce = 8;
  for (int64_t i = first + threadIdx.x; i < last; i += kAtOnce * kT) {
    int t[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) t[j] = i + j * kT < last ? tokens[i + j * kT] : -1;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (t[j] >= v0 && t[j] < v0 + kPromptSlice) atomicOr(&seen[(t[j] - v0) >> 5], 1u << (t[j] & 31));
  }
  __syncthreads();
  uint16_t* p = state + static_cast<int64_t>(r) * V;
  for (int i = threadIdx.x * 8; i < kPromptSlice && v0 + i < V; i += kT * 8) {
    const uint32_t b = seen[i >> 5] >> (i & 31);
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = (b >> (2 * e) & 1u) << 15 | (b >> (2 * e + 1) & 1u) << 31;
    store_words(p + v0 + i, min(8, V - v0 - i), w);
  }
}

// A wave a request, 64 tokens at a time; a token that is there several times is
// counted by the first lane that has it.
__global__ __launch_bounds__(kT) void logits_commit_kernel(int R, int gamma, int V, const int32_t* ell,
                                                           const int32_t* n_acc, const int32_t* x0, const int32_t* x,
                                                           uint16_t* state) {
  const int r = blockIdx.x * (kT / 64) + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (r >= R) return;
  const int rows = rows_of(ell[r], gamma);
  if (rows == 0) return;
  const int n = x ? min(max(n_acc[r], 0), rows - 1) + 1 : 1;
  uint16_t* p = state + static_cast<int64_t>(r) * V;
  for (int j0 = 0; j0 < n; j0 += 64) {
    const int j = j0 + lane;
    const int t = j >= n ? -1 : token_or_none(j == 0 ? x0[r] : x[static_cast<int64_t>(r) * gamma + j - 1], V);
    int times = 0;
    bool first = true;
    for (int l = 0; l < 64 && j0 + l < n; ++l) {
      const bool same = __builtin_amdgcn_readlane(t, l) == t;
      times += same;
      if (same && l < lane) first = false;
    }
    if (t >= 0 && first) {
      const uint32_t s = p[t];
      p[t] = static_cast<uint16_t>((s & kInPrompt) | min((s & kCount) + times, kCount));
    }
    __threadfence_block();  // the next 64 may count the same tokens
  }
}

}  // namespace

hipError_t logits_launch(dspark_dtype dt, int R, int gamma, int V, const void* logits, const int32_t* row0,
                         const int32_t* ell, const int32_t* x0, const int32_t* x, const uint16_t* state,
                         const float* repetition, const float* presence, const float* frequency, int nb,
                         const int32_t* bias_tok, const float* bias, const uint32_t* mask, void* out, hipStream_t s) {
  LogitsArgs a{R, gamma, V, nb, logits, row0, ell, x0, x, state, repetition, presence, frequency, bias_tok, bias,
               reinterpret_cast<const uint8_t*>(mask), 4LL * ceil_div(V, 32), out, 0};
  const int slices = ceil_div(V, kSlice);
  // rows of a request together (its counts and biases are loaded once), unless
  // that leaves compute units without work.  With the prompt and the commit, 4 x
  // 17 rows of 129280 take 11.8 us at 8 work groups a compute unit, 13.8 at 2,
  // 15.0 at 32, 32 x 9 of 50257 16.8, 19.2 and 20.5.
  const int64_t groups = static_cast<int64_t>(slices) * R, want = 8LL * compute_units();
  int parts = groups >= want ? 1 : static_cast<int>(want / groups);
  if (parts > gamma + 1) parts = gamma + 1;
  a.rows_each = ceil_div(gamma + 1, parts);
  const dim3 grid(slices, R, ceil_div(gamma + 1, a.rows_each));
  if (dt == DSPARK_F32) logits_kernel<float, Logits32><<<grid, kT, 0, s>>>(a);
  else logits_kernel<uint16_t, Logits16><<<grid, kT, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t logits_prompt_launch(int R, int V, int64_t n, const int32_t* tokens, const int32_t* start,
                                const int32_t* count, uint16_t* state, hipStream_t s) {
  logits_prompt_kernel<<<dim3(ceil_div(V, kPromptSlice), R), kT, 0, s>>>(V, n, tokens, start, count, state);
  return hipGetLastError();
}

hipError_t logits_commit_launch(int R, int gamma, int V, const int32_t* ell, const int32_t* n_acc, const int32_t* x0,
                                const int32_t* x, uint16_t* state, hipStream_t s) {
  logits_commit_kernel<<<ceil_div(R, kT / 64), kT, 0, s>>>(R, gamma, V, ell, n_acc, x0, x, state);
  return hipGetLastError();
}

}  // namespace dspark

using namespace dspark;

// ---------------------------------------------------------------- the C ABI

namespace {

bool shape_ok(int R, int gamma, int V) {
  return R >= 1 && R <= kCacheMaxR && gamma >= 0 && gamma <= kCacheMaxGamma && V >= 2 && V < (1 << 24);
}
bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
dspark_status launched(hipError_t e) { return e == hipSuccess ? DSPARK_OK : DSPARK_ELAUNCH; }

}  // namespace

extern "C" {

dspark_status dspark_logits(dspark_dtype dt, int R, int gamma, int V, const void* logits, const int32_t* row0,
                            const int32_t* ell, const int32_t* x0, const int32_t* x, const uint16_t* state,
                            const float* repetition, const float* presence, const float* frequency, int nb,
                            const int32_t* bias_tok, const float* bias, const uint32_t* mask, void* out,
                            void* stream) {
  if (dt != DSPARK_F32 && dt != DSPARK_BF16) return DSPARK_EDTYPE;
  if (!shape_ok(R, gamma, V) || nb < 0 || nb > (1 << 20)) return DSPARK_EINVAL;
  if (!logits || !ell || !out || (state && !x0) || (nb > 0 && (!bias_tok || !bias))) return DSPARK_EINVAL;
  if (!aligned16(logits) || !aligned16(out) || !aligned16(state)) return DSPARK_EINVAL;
  const dspark_status st = check_device();
  if (st != DSPARK_OK) return st;
  return launched(logits_launch(dt, R, gamma, V, logits, row0, ell, x0, x, state, repetition, presence, frequency, nb,
                                bias_tok, bias, mask, out, static_cast<hipStream_t>(stream)));
}

dspark_status dspark_logits_prompt(int R, int V, int64_t n, const int32_t* tokens, const int32_t* start,
                                   const int32_t* count, uint16_t* state, void* stream) {
  if (!shape_ok(R, 0, V) || n < 0 || n >= (1LL << 31)) return DSPARK_EINVAL;
  if ((n > 0 && !tokens) || !start || !count || !state || !aligned16(state)) return DSPARK_EINVAL;
  const dspark_status st = check_device();
  if (st != DSPARK_OK) return st;
  return launched(logits_prompt_launch(R, V, n, tokens, start, count, state, static_cast<hipStream_t>(stream)));
}

dspark_status dspark_logits_commit(int R, int gamma, int V, const int32_t* ell, const int32_t* n_acc,
                                   const int32_t* x0, const int32_t* x, uint16_t* state, void* stream) {
  if (!shape_ok(R, gamma, V)) return DSPARK_EINVAL;
  if (!ell || !n_acc || !x0 || !state || !aligned16(state)) return DSPARK_EINVAL;
  const dspark_status st = check_device();
  if (st != DSPARK_OK) return st;
  return launched(logits_commit_launch(R, gamma, V, ell, n_acc, x0, x, state, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
