// Log probabilities of given tokens, with the entropy, the token's rank and the
// top alternatives, and the gradient of the logits.  Per row of logits l, with
// M = max l, d = c (l - M) (c > 0), S = sum exp(d), T = sum exp(d) d:
//   logp = d_t - log S,  H = log S - T / S,  rank = #{l > l_t}
//   dl = c (g (1_t - p) - e p (log p + H)),  p = exp(d - log S)
// (l - M before the product with c: masks of the type's lowest value would
// overflow in c l, and a row of them would lose its maximum.)
// A logit of -inf is a masked token: probability 0, never an alternative.  A
// row of nothing else has logp -inf, entropy 0 and gradient 0.
//
// One pass over the logits.  A workgroup walks its part of a row in chunks
// that its threads hold in registers (32 to 128 bytes each), so the
// maximum, the sums under it and the search for alternatives read memory once.
// Every thread keeps its own running maximum and sums (no barrier between the
// maximum and the exponentials); they meet once per workgroup.
//
// Alternatives: a bound b that at least `top` logits reach turns the search
// into a collection of the few logits >= b.  For the first chunk b is the
// top-th largest of 64 group maxima (4 threads or 1); afterwards it is the
// last alternative of the list so far (later ids lose ties, so > b).  The
// candidates meet the list in LDS and each finds its place by counting the
// larger keys; keys (value, id) are distinct, so the order of arrival does not
// matter.  Where ties or an order against the walk give more candidates than
// the buffer holds, the chunk's alternatives are found one by one.
//
// With few rows, several workgroups share a row (arrival counters, the last
// one joins the parts in their order, so the sums do not depend on timing).
//
// Many rows are bound by their bytes: 2048 x 131072 bf16 (537 MB) in 101 us
// without alternatives and 114 us with 20 of them and a fifth of the tokens
// masked.  Rows that are short, or a few hundred, are not: every chunk ends in the
// chain that finds its alternatives before the next one is asked for, and a row a
// little longer than a chunk has the chain twice (us without / with 20
// alternatives, floor: 3963 x 4096 bf16 10.8 / 15.5, 6.4; 3963 x 4197 16.3 / 22.2,
// 6.6; 1000 x 12000 11.2 / 14.7, 4.7; 2000 x 16000 19.7 / 31.3, 12.6; 256 x 131072
// 21.7 / 29.7, 13.3).  One row of 131072 fp32 takes 11.4 us, a chain of latencies:
// 2.0 until its logits are there, 3.4 for the alternatives and sums of a part, 0.7
// to publish them, 1.3 for the last workgroup to read the parts, 2.7 to join them.
#include <hip/hip_runtime.h>

#include "qg_device.h"
#include "qg_internal.h"
#include "qg_mm.h"

namespace qg {

namespace {

constexpr int kThreads = 256;    // of a workgroup (or 64: one wave, see logprobs_split)
constexpr int kMaxParts = 64;    // workgroups per row
constexpr int kCounterPitch = 16;  // rows' arrival counters, 64 bytes apart: in one line they wait for each other
constexpr int kRecordKeys = kMaxParts * QG_MAX_ALTERNATIVES / kThreads;  // keys of a row's parts, per thread
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// Order of floats as unsigned numbers (no NaN), and back.
__device__ __forceinline__ uint32_t order_bits(float l) {
  const uint32_t u = __float_as_uint(l);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? u & 0x7FFFFFFFu : ~u);
}

// Order of alternatives as one key: larger logits first, equal ones by lower
// id (-0 equals +0).
__device__ __forceinline__ uint64_t alt_key(float l, uint32_t id) {
  return ((uint64_t)order_bits(l + 0.f) << 32) | (0xFFFFFFFFu - id);
}
__device__ __forceinline__ float key_value(uint64_t k) { return order_value((uint32_t)(k >> 32)); }
__device__ __forceinline__ int key_id(uint64_t k) { return (int)(0xFFFFFFFFu - (uint32_t)k); }

// The largest of three (a NaN loses against a number).  Written out because
// fmaxf first quiets every operand of unknown origin, an instruction each.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// The next number above l (the most negative one above -inf); l is no NaN.
__device__ __forceinline__ float next_above(float l) {
  const uint32_t u = __float_as_uint(l + 0.f);
  return u == 0x7F800000u ? l : __uint_as_float((u & 0x80000000u) ? u - 1 : u + 1);
}

// A number that at least `top` (<= 64) of the 64 lanes' u reach: the top-th
// largest with its low 12 bits cleared, found bit by bit from ballots.
__device__ __forceinline__ uint32_t wave_bound(uint32_t u, int top) {
  uint32_t bound = 0;
#pragma unroll
  for (int bit = 31; bit >= 12; --bit) {
    const uint32_t next = bound | (1u << bit);
    if (__popcll(__ballot(u >= next)) >= top) bound = next;
  }
  return bound;
}

// Running maximum and sums (log2 scale: the exponent is c2 (l - m))
struct Sums {
  float m, s, t;
};
// The sums under another maximum m (-inf: there is none).  t is in units of the
// exponent (base 2).
__device__ __forceinline__ Sums under(const Sums &a, float m, float c2) {
  const float d = fmaxf((a.m - (m == neg_inf() ? 0.f : m)) * c2, -200.f), f = __builtin_amdgcn_exp2f(d);
  return Sums{m, a.s * f, f * (a.t + d * a.s)};
}
// Reductions over a wave, the result in every lane: pairs, quads, 8 and 16
// lanes by data-parallel moves, then across the rows of 16.
template <int CTRL>
__device__ __forceinline__ int lanes_moved(int x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, 0xF, 0xF, true);
}
template <class V, class Op>
__device__ __forceinline__ V wave_reduce(V x, Op op) {
  auto moved = [](V v, auto ctrl) { return __builtin_bit_cast(V, lanes_moved<decltype(ctrl)::value>(__builtin_bit_cast(int, v))); };
  x = op(x, moved(x, std::integral_constant<int, 0xB1>{}));   // quad_perm 1 0 3 2
  x = op(x, moved(x, std::integral_constant<int, 0x4E>{}));   // quad_perm 2 3 0 1
  x = op(x, moved(x, std::integral_constant<int, 0x141>{}));  // row_half_mirror
  x = op(x, moved(x, std::integral_constant<int, 0x140>{}));  // row_mirror
  x = op(x, (V)__shfl_xor(x, 16));
  return op(x, (V)__shfl_xor(x, 32));
}
__device__ __forceinline__ Sums wave_sums(const Sums &a, float c2) {
  const auto add = [](float x, float y) { return x + y; };
  const float m = wave_reduce(a.m, [](float x, float y) { return fmaxf(x, y); });
  const Sums u = under(a, m, c2);
  return Sums{m, wave_reduce(u.s, add), wave_reduce(u.t, add)};
}

template <int T, int VEC, bool SHARED>
struct Shared {
  static constexpr int CAP = 4 * T;       // candidates of one chunk
  static constexpr int UNITS = 256;       // 16-byte units that hold them
  static constexpr bool DATA = VEC <= 2;  // units by value (else read again)
  static constexpr int KEYS = SHARED ? kMaxParts * QG_MAX_ALTERNATIVES : CAP;
  static_assert(CAP <= KEYS, "candidate buffer");
  uint64_t cand[KEYS + QG_MAX_ALTERNATIVES + 8];
  uint64_t list[QG_MAX_ALTERNATIVES];
  u32x4 unit[DATA ? UNITS : 1];
  int place[UNITS];
  float group[64];
  Sums sums[T / 64];
  uint64_t best[T / 64];
  int above[T / 64];
  int count, units;
  int flag;
};

}  // namespace

template <bool F32, int VEC, int T>
struct Chunk {
  static constexpr int EPV = F32 ? 4 : 8;            // logits per 16 bytes
  static constexpr int EL = F32 ? 4 : 2;
  static constexpr uint32_t NONE = F32 ? 0xFF800000u : 0xFF80FF80u;  // -inf
  static constexpr int SIZE = T * VEC * EPV;  // logits per chunk
  u32x4 d[VEC];

  // Chunk at logit `first` of a row of `vocab`.  16 bytes that the row's end
  // cuts are read whole, ending with the row, and what is the neighbour's of
  // them is masked; so is everything behind the end.
  __device__ __forceinline__ void load(const uint8_t *row, int first, int base, int vocab, bool once) {
    if (first + SIZE <= vocab) {
      if (once) {
        asm volatile("");  // (else both branches become one, of plain loads)
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          d[v] = __builtin_nontemporal_load((const u32x4_any *)(row + (int64_t)place(base, v) * EL));
        asm volatile("");
        return;
      }
#pragma unroll
      for (int v = 0; v < VEC; ++v) d[v] = *(const u32x4_any *)(row + (int64_t)place(base, v) * EL);
      return;
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) load16(v, row, place(base, v), vocab);
  }
  // the 16 bytes of logits i ..
  __device__ __forceinline__ void load16(int v, const uint8_t *row, int i, int vocab) {
    d[v] = u32x4{NONE, NONE, NONE, NONE};
    if (i >= vocab) return;
    if (vocab < EPV) {  // (a row of less than 16 bytes: i is 0)
      for (int e = 0; e < vocab; ++e) set(v, e, F32 ? ((const uint32_t *)row)[e] : ((const uint16_t *)row)[e]);
      return;
    }
    const int at = min(i, vocab - EPV);
    d[v] = *(const u32x4_any *)(row + (int64_t)at * EL);
    if (at < i) {
#pragma unroll
      for (int e = 0; e < EPV - 1; ++e)
        if (at + e < i) set(v, e, NONE);
    }
  }
  // replaces one logit by its bits (the low ones of `bits`)
  __device__ __forceinline__ void set(int v, int e, uint32_t bits) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if constexpr (F32)
        d[v][w] = w == e ? bits : d[v][w];
      else if (w == e >> 1)
        d[v][w] = (e & 1) ? (d[v][w] & 0xFFFFu) | (bits << 16) : (d[v][w] & 0xFFFF0000u) | (bits & 0xFFFFu);
    }
  }
  __device__ __forceinline__ float at(int v, int e) const {
    if constexpr (F32)
      return __uint_as_float(d[v][e]);
    else
      return __uint_as_float((e & 1) ? d[v][e / 2] & 0xFFFF0000u : d[v][e / 2] << 16);
  }
  // The thread's place in a chunk at `first` (16 bytes of every thread, then the
  // next of every thread: a row that fills a part of the chunk still gives every
  // group of threads a maximum and every wave work), opaque to the compiler: it
  // would keep everything that follows from it for every v, in a register each.
  __device__ __forceinline__ static int base_of(int first) {
    int base = first + (int)threadIdx.x * EPV;
    asm volatile("" : "+v"(base));
    return base;
  }
  // first logit of its v-th 16 bytes: their place, and where they were read
  __device__ __forceinline__ static int place(int base, int v) { return base + v * T * EPV; }
  __device__ __forceinline__ static int id(int base, int v, int vocab) {
    return max(min(place(base, v), vocab - EPV), 0);
  }
};

// Merges sh.cand[0 .. n) and sh.list[0 .. have) into sh.list; returns its
// length.  All threads call; the candidates are visible before the call.
template <int T, int VEC, bool SHARED>
__device__ __forceinline__ int merge_list(Shared<T, VEC, SHARED> &sh, int n, int have, int top) {
  const int all = n + have;
  // (zeros, below every key, to a multiple of 8)
  for (int i = threadIdx.x; i < have + 8; i += T) sh.cand[n + i] = i < have ? sh.list[i] : 0;
  __syncthreads();
  for (int i = threadIdx.x; i < all; i += T) {
    const uint64_t k = sh.cand[i];
    int r = 0;
    for (int j0 = 0; j0 < all; j0 += 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) r += sh.cand[j0 + j] > k;
    }
    if (r < top) sh.list[r] = k;
  }
  __syncthreads();
  return min(all, top);
}

// The chunk's part in the list of alternatives; vmax: the largest logit of
// each of the thread's 16 bytes, most: of all.  Uniform over the workgroup;
// returns the list's length.
template <bool F32, int VEC, int T, bool SHARED>
__device__ __forceinline__ int take_alternatives(Shared<T, VEC, SHARED> &sh, const Chunk<F32, VEC, T> &ch, const float (&vmax)[VEC],
                                                 const uint8_t *row, int vocab, int first, float most, int have,
                                                 int top) {
  using C = Chunk<F32, VEC, T>;
  using S = Shared<T, VEC, SHARED>;
  const float last = have == top ? key_value(sh.list[top - 1]) : neg_inf();
  if (!__syncthreads_or(most > last)) return have;
  float bound = next_above(last);  // candidates: l >= bound
  for (int attempt = have == top ? 0 : 1; attempt < 2; ++attempt) {
    if (attempt == 1) {
      // what `top` of the 64 group maxima reach
      // (of the first wave's threads where they hold everything)
      float g = most;
      const int per = vocab - first <= 64 * C::EPV ? 1 : T / 64;
      for (int off = 1; off < per; off <<= 1) g = fmaxf(g, __shfl_xor(g, off));
      if (threadIdx.x % per == 0 && threadIdx.x < 64 * per) sh.group[threadIdx.x / per] = g;
      __syncthreads();
      bound = fmaxf(bound, order_value(max(wave_bound(order_bits(sh.group[threadIdx.x & 63]), top),
                                           order_bits(-3.402823466e38f))));
    }
    if (threadIdx.x == 0) sh.count = sh.units = 0;
    __syncthreads();
    // the few 16-byte units that hold candidates, then their logits, one per
    // thread: short code (unrolled over a thread's logits, fetching the
    // instructions took longer than anything else)
    const int base = C::base_of(first);
    uint32_t hit = 0;
#pragma unroll
    for (int v = 0; v < VEC; ++v) hit |= vmax[v] >= bound ? 1u << v : 0u;
    if (hit != 0) {
      int at = atomicAdd(&sh.units, __popc(hit));
      if constexpr (S::DATA) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          if ((hit >> v & 1u) == 0 || at >= S::UNITS) continue;
          sh.place[at] = C::place(base, v);
          sh.unit[at++] = ch.d[v];
        }
      } else {
        for (; hit != 0 && at < S::UNITS; hit &= hit - 1) sh.place[at++] = C::place(base, __ffs(hit) - 1);
      }
    }
    __syncthreads();
    const int units = sh.units;
    if (units <= S::UNITS) {
      for (int i = threadIdx.x; i < units * C::EPV; i += T) {
        const int u = i / C::EPV, e = i % C::EPV, from = sh.place[u], id = max(min(from, vocab - C::EPV), 0) + e;
        float l = neg_inf();
        if constexpr (S::DATA)
          l = F32 ? ((const float *)&sh.unit[u])[e] : bf16_bits_to_f32(((const uint16_t *)&sh.unit[u])[e]);
        else if (id >= from && id < vocab)
          l = F32 ? ((const float *)row)[id] : bf16_bits_to_f32(((const uint16_t *)row)[id]);
        if (l >= bound) {
          const int at = atomicAdd(&sh.count, 1);
          if (at < S::CAP) sh.cand[at] = alt_key(l, (uint32_t)id);
        }
      }
      __syncthreads();
      const int n = sh.count;
      if (n <= S::CAP) return merge_list(sh, n, have, top);
    }
    __syncthreads();  // (the counts are cleared for the next attempt)
  }
  // one by one: the largest key below the one before it
  int n = 0;
  for (uint64_t below = ~0ull; n < top; ++n) {
    uint64_t best = 0;
    for (int i = first + (int)threadIdx.x; i < min(first + C::SIZE, vocab); i += T) {  // (read again: rare)
      const float l = F32 ? ((const float *)row)[i] : bf16_bits_to_f32(((const uint16_t *)row)[i]);
      const uint64_t k = alt_key(l, (uint32_t)i);
      if (l > last && k < below && k > best) best = k;
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint64_t o = __shfl_xor((unsigned long long)best, off);
      best = o > best ? o : best;
    }
    if ((threadIdx.x & 63) == 0) sh.best[threadIdx.x >> 6] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < T / 64; ++w) best = sh.best[w] > best ? sh.best[w] : best;
    __syncthreads();
    if (best == 0) break;  // uniform
    if (threadIdx.x == 0) sh.cand[n] = best;
    below = best;
  }
  __syncthreads();
  return merge_list(sh, n, have, top);
}

// The record of one part of a row: sums, count and the sorted alternatives.
__host__ __device__ constexpr int64_t record_bytes(int top) { return 16 + 8 * (int64_t)((top + 1) & ~1); }

// SHARED: gridDim.x workgroups share a row.  T: threads of a workgroup.
template <bool F32, int VEC, bool SHARED, int T = kThreads>
__global__ __launch_bounds__(T, SHARED ? 4 : 5) void logprobs_kernel(LogprobArgs a, uint32_t *counters, uint8_t *records) {
  using C = Chunk<F32, VEC, T>;
  __shared__ Shared<T, VEC, SHARED> sh;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int vocab = (int)a.vocab;
  const float c2 = a.scale * kLog2e;
  const int parts = SHARED ? gridDim.x : 1, part = SHARED ? blockIdx.x : 0;
  // Logits that the last-level cache (256 MB) does not hold and that no gradient
  // reads again (no statistics are asked for) are read past the caches: 2048 x
  // 131072 bf16 (537 MB), written just before, 314 us for both against 336, 512 x
  // 131072 fp32 (268 MB) 152 against 159.  Smaller ones are found there, as the
  // head layer wrote them: past the caches 256 x 131072 bf16 (67 MB) 54.8 against
  // 48.3, 4000 x 8192 49.4 against 42.5, 64 x 131072 23.3 against 22.0.  (A reader
  // behind it costs large ones what they gain: 214 against 205; a gradient more,
  // 1021 x 100003 bf16 136 against 119.)
  const bool once = a.stats == nullptr && a.rows * a.vocab * (F32 ? 4 : 2) >= (256ll << 20);
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const uint8_t *lp = (const uint8_t *)a.logits + row * a.ldl * (F32 ? 4 : 2);
    // this workgroup's logits, in equal parts (a short last one would have no
    // good bound for its alternatives, and the others would wait for it)
    const int64_t all_units = (vocab + C::EPV - 1) / C::EPV;
    const int begin = SHARED ? (int)(part * all_units / parts) * C::EPV : 0;
    const int end = SHARED ? min((int)((part + 1) * all_units / parts) * C::EPV, vocab) : vocab;
    // the first chunk is asked for ahead of the token and its logit, which take
    // two trips to memory (with 8 units that would cost a wave's registers)
    constexpr bool AHEAD = VEC <= 4;
    C ch;
    if constexpr (AHEAD) {
      ch.load(lp, begin, C::base_of(begin), end, once);
      __builtin_amdgcn_sched_barrier(0);
    }
    const int tok = a.tokens ? a.tokens[row] : -1;
    const bool in = tok >= 0 && tok < vocab;
    const float lt = !in ? __builtin_inff()
                     : F32 ? ((const float *)lp)[tok] : bf16_bits_to_f32(((const uint16_t *)lp)[tok]);
    Sums st = {neg_inf(), 0.f, 0.f};
    int above = 0, have = 0;
    for (int first = begin; first < end; first += C::SIZE) {
      if (!AHEAD || first > begin) ch.load(lp, first, C::base_of(first), end, once);
      float most = neg_inf(), vmax[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        vmax[v] = neg_inf();
#pragma unroll
        for (int e = 0; e < C::EPV; e += 2) vmax[v] = max3(vmax[v], ch.at(v, e), ch.at(v, e + 1));
        most = fmaxf(most, vmax[v]);
      }
      // the running sums under the new maximum
      const float m = fmaxf(st.m, most);
      const float base = m == neg_inf() ? 0.f : m;
      const float back = fmaxf((st.m - base) * c2, -200.f), f = __builtin_amdgcn_exp2f(back);
      float s = st.s * f, t = f * (st.t + back * st.s);
      int hits = 0;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        // one 16 bytes after the other: unpacked again (an instruction per
        // logit) instead of held in a register per logit, their masks counted
        // before the next ones are made
        asm volatile("" : "+v"(ch.d[v]), "+v"(s), "+v"(t), "+s"(hits));
#pragma unroll
        for (int e = 0; e < C::EPV; ++e) {
          const float l = ch.at(v, e);
          const float d = (l - base) * c2, x = __builtin_amdgcn_exp2f(d);
          s += x;
          t = __builtin_fmaf(x, fmaxf(d, -200.f), t);  // (0 * -inf for masked tokens; a NaN comes in through x)
          hits += __popcll(__ballot(l > lt));          // wave-uniform
        }
      }
      st = Sums{m, s, t};
      above += hits;
      if (a.top > 0) have = take_alternatives<F32, VEC, T, SHARED>(sh, ch, vmax, lp, end, first, most, have, a.top);
    }
    // join the threads, then the waves
    st = wave_sums(st, c2);
    if (lane == 0) {
      sh.sums[wave] = st;
      sh.above[wave] = above;
    }
    __syncthreads();
    {
      float m = neg_inf();
#pragma unroll
      for (int w = 0; w < T / 64; ++w) m = fmaxf(m, sh.sums[w].m);
      st = Sums{m, 0.f, 0.f};
      above = 0;
#pragma unroll
      for (int w = 0; w < T / 64; ++w) {
        const Sums u = under(sh.sums[w], m, c2);
        st.s += u.s;
        st.t += u.t;
        above += sh.above[w];
      }
    }
    if constexpr (SHARED) {
      // publish this part, and let the last workgroup of the row join them:
      // agent-scope stores, complete before the counter moves
      const int64_t rb = record_bytes(a.top);
      uint8_t *rec = records + row * parts * rb;
      float *rf = (float *)(rec + part * rb);
      if (threadIdx.x < 4) {
        const float v = threadIdx.x == 0 ? st.m : threadIdx.x == 1 ? st.s : threadIdx.x == 2 ? st.t : __int_as_float(above);
        __hip_atomic_store(rf + threadIdx.x, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      if ((int)threadIdx.x < a.top)
        __hip_atomic_store((uint64_t *)(rf + 4) + threadIdx.x, (int)threadIdx.x < have ? sh.list[threadIdx.x] : 0ull,
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      if (threadIdx.x == 0)
        sh.flag = __hip_atomic_fetch_add(counters + row * kCounterPitch, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                  (uint32_t)(parts - 1);
      __syncthreads();
      if (!sh.flag) {  // uniform over the workgroup
        __syncthreads();
        continue;
      }
      auto word = [&](int p, int i) {
        return __hip_atomic_load((const float *)(rec + p * rb) + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      };
      auto key = [&](int p, int i) {
        return __hip_atomic_load((const uint64_t *)(rec + p * rb + 16) + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      };
      // every load of the records goes out at once: this thread's keys (one
      // position of a list each), this lane's sums
      uint64_t all[kRecordKeys], mine = 0;
      if (a.top > 0) {
        const int deep = (a.top + parts - 1) / parts;
        mine = lane < parts * deep ? key(lane % parts, lane / parts) : 0;
#pragma unroll
        for (int j = 0; j < kRecordKeys; ++j) {
          const int i = j * kThreads + (int)threadIdx.x, pos = i / kMaxParts, p = i % kMaxParts;
          all[j] = pos < a.top && p < parts ? key(p, pos) : 0;
        }
      }
      st = Sums{neg_inf(), 0.f, 0.f};
      above = 0;
      if (lane < parts) {
        st = Sums{word(lane, 0), word(lane, 1), word(lane, 2)};
        above = __float_as_int(word(lane, 3));
      }
      st = wave_sums(st, c2);
      above = wave_reduce(above, [](int x, int y) { return x + y; });
      if (a.top > 0) {
        // the first `deep` keys of each list (`mine`) are at least `top` keys: what `top`
        // of their values reach bounds the list (ties and all, the buffer holds
        // every key of every part)
        const uint64_t bound = (uint64_t)wave_bound((uint32_t)(mine >> 32), a.top) << 32;
        if (threadIdx.x == 0) sh.count = 0;
        __syncthreads();
        int n = 0;
#pragma unroll
        for (int j = 0; j < kRecordKeys; ++j) n += all[j] != 0 && all[j] >= bound;
        if (n > 0) {
          int at = atomicAdd(&sh.count, n);
#pragma unroll
          for (int j = 0; j < kRecordKeys; ++j)
            if (all[j] != 0 && all[j] >= bound) sh.cand[at++] = all[j];
        }
        __syncthreads();
        have = merge_list(sh, sh.count, 0, a.top);
      }
      if (threadIdx.x == 0) __hip_atomic_store(counters + row * kCounterPitch, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    const bool empty = st.m == neg_inf() && st.s == 0.f;
    const float most = st.m == neg_inf() ? 0.f : st.m;
    const float log_s = empty ? neg_inf() : logf(st.s);
    if (threadIdx.x == 0) {
      if (a.logp) a.logp[row] = !in ? __builtin_nanf("") : empty ? neg_inf() : (lt - most) * a.scale - log_s;
      if (a.rank) a.rank[row] = in ? above : -1;
      if (a.entropy) a.entropy[row] = empty ? 0.f : log_s - st.t / st.s * kLn2;
      if (a.stats) {
        a.stats[2 * row] = most;
        a.stats[2 * row + 1] = log_s;
      }
    }
    if ((int)threadIdx.x < a.top) {
      const bool there = (int)threadIdx.x < have;
      const uint64_t k = there ? sh.list[threadIdx.x] : 0;
      if (a.top_ids) a.top_ids[row * a.top + threadIdx.x] = there ? key_id(k) : -1;
      if (a.top_logp)
        a.top_logp[row * a.top + threadIdx.x] = there ? (key_value(k) - most) * a.scale - log_s : neg_inf();
    }
    __syncthreads();  // sh is used again for the next row
  }
}

// dl in one pass: 16 bytes per thread and step, VEC steps of a row in flight.
// Reads and writes of one 16 bytes are the same thread's, so dl may be l.  From
// the last row on: what the forward pass read last is found in the caches
// (forward and backward of 2048 x 131072 bf16: 334 -> 330 us).  PAST: a gradient
// larger than the L2s (32 MB) is written past the caches, where it would push
// out the logits and be written back behind the next reads (forward and backward
// of 1021 x 100003 bf16 140 -> 121 us); a smaller one stays for who reads it next.
// Bound by its bytes.
template <bool F32, int VEC, bool PAST>
__global__ __launch_bounds__(kThreads) void logprobs_backward_kernel(LogprobArgs a) {
  using C = Chunk<F32, VEC, kThreads>;
  constexpr int EL = F32 ? 4 : 2;
  const int vocab = (int)a.vocab;
  const float c2 = a.scale * kLog2e;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const int64_t row = a.rows - 1 - r;
    const uint8_t *lp = (const uint8_t *)a.logits + row * a.ldl * EL;
    uint8_t *dp = (uint8_t *)a.dlogits + row * a.lddl * EL;
    const float most = a.stats[2 * row], log_s = a.stats[2 * row + 1];
    const bool empty = log_s == neg_inf();
    const int tok = a.tokens ? a.tokens[row] : -1;
    const float g = a.dlogp && tok >= 0 && tok < vocab && !empty ? a.dlogp[row] * a.scale : 0.f;
    const float e = a.dentropy && !empty ? a.dentropy[row] * a.scale : 0.f;
    // -p (g + e (log p + H)) = p (w0 - e ln2 q) with q = log2 p
    const float w0 = -g - (e != 0.f ? e * a.entropy[row] : 0.f), w1 = -e * kLn2, q0 = empty ? 0.f : -log_s * kLog2e;
    for (int first = (int)blockIdx.x * C::SIZE; first < vocab; first += (int)gridDim.x * C::SIZE) {
      C ch;
      const int base = C::base_of(first);
      ch.load(lp, first, base, vocab, false);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const int i = C::place(base, v), at = C::id(base, v, vocab);
        float o[C::EPV];
#pragma unroll
        for (int k = 0; k < C::EPV; ++k) {
          const float q = __builtin_fmaf(ch.at(v, k) - most, c2, q0);
          o[k] = __builtin_amdgcn_exp2f(q) * __builtin_fmaf(w1, fmaxf(q, -300.f), w0);
          if (at + k == tok) o[k] += g;
        }
        u32x4 w;
        if constexpr (F32) {
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = __float_as_uint(o[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = bf16_rne(o[2 * k]) | (bf16_rne(o[2 * k + 1]) << 16);
        }
        if (empty) w = u32x4{0u, 0u, 0u, 0u};
        if (i + C::EPV <= vocab) {
          if constexpr (PAST)
            __builtin_nontemporal_store(w, (u32x4_any *)(dp + (int64_t)i * EL));
          else
            *(u32x4_any *)(dp + (int64_t)i * EL) = w;
        } else {
          uint8_t *p = dp + (int64_t)at * EL;
#pragma unroll
          for (int k = 0; k < C::EPV; ++k) {
            if (at + k < i || at + k >= vocab) continue;
            if constexpr (F32)
              ((uint32_t *)p)[k] = w[k];
            else
              ((uint16_t *)p)[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
          }
        }
      }
    }
  }
}

namespace {
static_assert(768 * kCounterPitch * 4 <= kSplitCounterBytes, "counters of shared rows");
// 16-byte units per thread and chunk, workgroups per row and their threads.  A
// row that one chunk holds takes the smallest that does and one workgroup (19
// rows of 6201 fp32: 9.3 us, 14.0 with smaller chunks that workgroups share);
// from 1024 of them on, which fill the CUs, one wave, so that no row waits at
// barriers (3963 rows of 4197 bf16: 22 us against 34; 1000 rows of 12000 bf16:
// 24 against 17).  Longer ones take the largest, or the smallest where the large
// chunks would leave CUs without a workgroup, and are shared by so many
// workgroups that each CU gets about three (at most one chunk each, kMaxParts).
struct Split {
  int vec, parts, threads;
};
Split logprobs_split(int64_t rows, int64_t vocab, bool f32) {
  const int64_t unit = (f32 ? 4 : 8) * kThreads;  // logits per unit of a chunk
  if (vocab <= 8 * unit) return Split{vocab <= 2 * unit ? 2 : vocab <= 4 * unit ? 4 : 8, 1, rows >= 1024 ? 64 : kThreads};
  const int vec = rows * ((vocab + 8 * unit - 1) / (8 * unit)) < 256 ? 2 : 8;
  const int64_t chunks = (vocab + vec * unit - 1) / (vec * unit), want = (768 + rows - 1) / rows;
  return Split{vec, (int)std::min<int64_t>(std::min<int64_t>(want, chunks), kMaxParts), kThreads};
}
}  // namespace

uint64_t logprobs_ws_bytes(int64_t rows, int64_t vocab, int top) {
  if (rows <= 0 || vocab <= 0) return 0;
  uint64_t b = 0;
  for (bool f32 : {false, true}) {
    const Split s = logprobs_split(rows, vocab, f32);
    if (s.parts > 1) b = std::max<uint64_t>(b, kSplitCounterBytes + align_up((uint64_t)(rows * s.parts * record_bytes(top)), 256));
  }
  return b;
}

hipError_t launch_logprobs(const LogprobArgs &a, void *ws, hipStream_t s) {
  const Split sp = logprobs_split(a.rows, a.vocab, a.f32);
  const dim3 grid((unsigned)sp.parts, (unsigned)std::min<int64_t>(a.rows, 65535));
  uint32_t *counters = (uint32_t *)ws;  // one per row: shared rows are fewer than 768
  uint8_t *records = (uint8_t *)ws + kSplitCounterBytes;
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(sp.threads), 0, s, a, counters, records); };
  auto typed = [&](auto f32) {
    constexpr bool F = decltype(f32)::value;
    if (sp.parts > 1)
      sp.vec == 2 ? go(logprobs_kernel<F, 2, true>) : go(logprobs_kernel<F, 8, true>);
    else if (sp.threads == 64)
      go(logprobs_kernel<F, 8, false, 64>);
    else
      sp.vec == 2 ? go(logprobs_kernel<F, 2, false>) : sp.vec == 4 ? go(logprobs_kernel<F, 4, false>) : go(logprobs_kernel<F, 8, false>);
  };
  a.f32 ? typed(std::true_type{}) : typed(std::false_type{});
  return hipGetLastError();
}

hipError_t launch_logprobs_backward(const LogprobArgs &a, hipStream_t s) {
  const int64_t size = (a.f32 ? 4 : 8) * kThreads * 4;
  const int64_t chunks = (a.vocab + size - 1) / size;
  // one workgroup per chunk up to about eight per CU, then more chunks each
  const int parts = (int)std::max<int64_t>(1, std::min<int64_t>(chunks, (2048 + a.rows - 1) / a.rows));
  const dim3 grid((unsigned)parts, (unsigned)std::min<int64_t>(a.rows, 65535));
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(kThreads), 0, s, a); };
  const bool past = a.rows * a.vocab * (a.f32 ? 4 : 2) > (32 << 20);
  if (a.f32)
    past ? go(logprobs_backward_kernel<true, 4, true>) : go(logprobs_backward_kernel<true, 4, false>);
  else
    past ? go(logprobs_backward_kernel<false, 4, true>) : go(logprobs_backward_kernel<false, 4, false>);
  return hipGetLastError();
}

}  // namespace qg
