// falcon_delta.hip - forward of the gated delta rule over a sequence (falcon_delta.h).
//
// A first launch forms every chunk's T (falcon_delta_solve.hip), a second walks: a workgroup has
// ND waves of 16 value rows each (falcon_delta_walk.h) and 2 ND waves beside them, which bring keys,
// q and gates, form the decayed scores and, one chunk behind, o^T = e (S q^T) + U^T P^T from the
// state's and u's operands that the walkers leave in LDS.  The outputs so come from operands that
// exist anyway, and u never goes to memory.
//
// 8x12x2048x64 bf16: 21 + 75 us of kernels, 90-99 us a call; memory would take 25 us (the walk
// moves 128 MB over the fabric).  Bound by the walk's latency: 32 chunks in order on 192 workgroups.
// 1x4x32771x128 in 16 segments: T 23, segments' writes 104, joins 27, walk 117 us (walked whole 1985 us).
// Not built, for their traffic: u written to memory and the outputs in a launch of their own (2.3
// times as much); T (b V) and T (b e K) formed beforehand in place of T, which shortens the chain by 12
// matrix instructions and one split and costs 40 KB a chunk.  Tried: half the output waves (us of
// the walk: 105 against 77); output waves that branch on their token tiles instead of having them as
// constants (107 against 105).
#include "falcon_delta_walk.h"

namespace falcon {
namespace delta {
namespace {

struct WalkArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* beta;
  const float* log_a;      // or null
  const uint4* T;
  const float* S0;         // or null
  float* o;
  float* S_out;            // or null; may be S0
  float* starts;           // [chain][segs][dv][dk]: slot j + 1 first segment j's own write,
                           // then slot j the state that segment j starts from
  uint4* moves;            // [chain][segs][StateT::kMove]: what a segment multiplies its start's rows with
  long chains;
  int seqlen, nv;
  int segs, per;           // segments of a chain, chunks of one
};

template <typename T, int DK, int ND>
struct WalkLds : StateLds<T, DK> {
  alignas(16) uint4 s[2][ND][StateLds<T, DK>::NQ][3][64];     // S at the chunk's start, as operands
  // U: as it is, for the output waves to split; at 128 columns, where they have more to do than
  // the state waves, as operands (us of the kernel: 1x4x32771x128 118 against 134, 8x12x2048x64
  // 79 against 75)
  static constexpr bool kSplit = DK == 128;
  alignas(16) uint4 u[2][ND][kSplit ? 6 : 4][64];
};

// Output waves of a workgroup of ND state waves, and the token tiles of output wave w.  (Waves
// go to the compute unit's four SIMDs in turn: with ND = 2 the tiles of most scores get the
// SIMDs without a state wave.)
constexpr int out_waves(int nd) { return 2 * nd; }
template <int ND>
__device__ __forceinline__ constexpr int tile_of(int w, int n) {
  return ND == 1 ? (n == 0 ? w : 3 - w) : w < 2 ? 3 - w : w - 2;
}

// The other waves: K and gates ahead, and the outputs of the chunk before.
template <typename T, int DK, int ND, int ow>
__device__ __forceinline__ void outputs(const WalkArgs& a, WalkLds<T, DK, ND>& lds, long chain, long c0, int n,
                                        int row0) {
  constexpr int NP = planes<T>(), NQ = (DK + 31) / 32, NTO = 64 * out_waves(ND), NT_ = 4 / out_waves(ND);
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const long len = a.seqlen, left = len - c0 * C;
  const T* q = static_cast<const T*>(a.q) + (chain * len + c0 * C) * DK;
  float* o = a.o + (chain * len + c0 * C) * a.nv + row0;
  Keys<T, DK, NTO, false> keys(lds, static_cast<const T*>(a.k) + (chain * len + c0 * C) * DK,
                               a.log_a ? a.log_a + chain * len + c0 * C : nullptr, a.beta + chain * len + c0 * C, left,
                               n, threadIdx.x - 64 * ND);
  constexpr int D = keys.D, R = keys.R;
  bf16x8 qf[NT_][NQ][NP], pf[NT_][2][3];
  float ev[NT_];
  PairRow<T, DK> qr[NT_];
  auto load_q = [&](int c) {
    const Window wq(q + (long)c * C * DK, left - (long)c * C, DK, 0);
#pragma unroll
    for (int j = 0; j < NT_; ++j) qr[j].load(wq, 16 * tile_of<ND>(ow, j) + m);
  };
  load_q(0);
#pragma unroll
  for (int j = 0; j < NT_; ++j) {
    ev[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int p = 0; p < NP; ++p) qf[j][i][p] = zero_frag();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int p = 0; p < 3; ++p) pf[j][i][p] = zero_frag();
  }
  // No branch in a step: one would make a wait for a load wait for the stores behind it.  Before
  // the first chunk the outputs go to a window of no rows, behind the last one K, q and the scores
  // are formed once more.
  for (int c = 0; c <= n; ++c) {
    __syncthreads();
    const int cc = c < n ? c : n - 1, ahead = c + D < n ? c + D : n - 1;
    keys.load(ahead);
    {
      const int b = (c + 1) & 1;
      const Window wo(o + (long)(c - 1) * C * a.nv, c > 0 ? left - (long)(c - 1) * C : 0, a.nv, c > 0 ? row0 : 0);
#pragma unroll
      for (int z = 0; z < ND; ++z) {
        floatx4 acc[NT_];
#pragma unroll
        for (int j = 0; j < NT_; ++j) acc[j] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          bf16x8 s[3];
#pragma unroll
          for (int p = 0; p < 3; ++p) s[p] = __builtin_bit_cast(bf16x8, lds.s[b][z][i][p][lane]);
#pragma unroll
          for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int r = 0; r < NP; ++r)
              if (p + r < 3) {
#pragma unroll
                for (int j = 0; j < NT_; ++j) acc[j] = mfma16(s[p], qf[j][i][r], acc[j]);
              }
        }
#pragma unroll
        for (int j = 0; j < NT_; ++j) acc[j] *= ev[j];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 1 && tile_of<ND>(ow, NT_ - 1) < 2) continue;
          bf16x8 u[3];
          if constexpr (WalkLds<T, DK, ND>::kSplit) {
#pragma unroll
            for (int p = 0; p < 3; ++p) u[p] = __builtin_bit_cast(bf16x8, lds.u[b][z][3 * i + p][lane]);
          } else {
            frag_pair(__builtin_bit_cast(floatx4, lds.u[b][z][2 * i][lane]),
                      __builtin_bit_cast(floatx4, lds.u[b][z][2 * i + 1][lane]), u);
          }
#pragma unroll
          for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int r = 0; p + r < 3; ++r)
#pragma unroll
              for (int j = 0; j < NT_; ++j)
                if (i == 0 || tile_of<ND>(ow, j) >= 2) acc[j] = mfma16(u[p], pf[j][i][r], acc[j]);
        }
#pragma unroll
        for (int j = 0; j < NT_; ++j) {
          // (2: past the caches)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uint4_t, acc[j]), wo.r,
                                                 ((16 * tile_of<ND>(ow, j) + m) * a.nv + 16 * z + 4 * g) * 4, 0, 2);
        }
      }
    }
    {
      // this chunk's scores, decayed: operands with rows t and slots s
      const uint16_t* kl = lds.k[cc % R][0];
      const Gates& gt = lds.gate[cc % R];
#pragma unroll
      for (int j = 0; j < NT_; ++j) {
        const int ti = tile_of<ND>(ow, j);
#pragma unroll
        for (int i = 0; i < NQ; ++i) qr[j].frag(i, qf[j][i]);
        ev[j] = gt.e[16 * ti + m];
        const float2 Gt = gt.g[16 * ti + m];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (2 * h > ti) continue;
          floatx4 p[2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int si = 2 * h + z;
            p[z] = floatx4{0.f, 0.f, 0.f, 0.f};
            if (si > ti) continue;
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
              bf16x8 kf[NP];
              pair_frag<NP, DK>(kl, 16 * si + m, i, kf);
              mma<NP, NP>(kf, qf[j][i], p[z]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float x = p[z][r] * decay(Gt, gt.g[16 * si + 4 * g + r]);
              p[z][r] = (si < ti || 4 * g + r <= m) ? x : 0.0f;
            }
          }
          frag_pair(p[0], p[1], pf[j][h]);
        }
      }
      load_q(c + 1 < n ? c + 1 : n - 1);
    }
    keys.store(lds, c + D);
  }
}

// The segment's outputs that are not finite formed anew, by the recurrence itself, one token
// at a time: a product over a chunk's tokens multiplies those that a mask leaves out with 0,
// and 0 * NaN is NaN, so that a NaN in v would reach every output of its chunk, also of
// earlier tokens.  The state behind the segment is not finite either, which is where it is
// looked for.  A row of the state lies on 8 lanes.
template <typename T, int DK, int ND>
__device__ __forceinline__ void walk_again(const WalkArgs& a, long chain, int seg, int row0) {
  constexpr int TPR = 8, N = DK / TPR;
  const long len = a.seqlen, state = (long)a.nv * DK, first = (long)seg * a.per * C;
  const long end = first + (long)a.per * C < len ? first + (long)a.per * C : len;
  const int row = row0 + (int)threadIdx.x / TPR, c0 = ((int)threadIdx.x % TPR) * N;
  const T* k = static_cast<const T*>(a.k) + chain * len * DK + c0;
  const T* q = static_cast<const T*>(a.q) + chain * len * DK + c0;
  const T* v = static_cast<const T*>(a.v) + chain * len * a.nv + row;
  const float* la = a.log_a ? a.log_a + chain * len : nullptr;
  const float* be = a.beta + chain * len;
  float* out = a.o + chain * len * a.nv + row;
  const float* S0 = a.segs > 1 ? a.starts + (chain * a.segs + seg) * state : a.S0 ? a.S0 + chain * state : nullptr;
  const long at = (long)row * DK + c0;
  float S[N];
#pragma unroll
  for (int j = 0; j < N; ++j) S[j] = S0 ? S0[at + j] : 0.0f;
  for (long t = first; t < end; ++t) {
    const float d = la ? exp2_of(log2_decay(la[t])) : 1.0f, b = be[t], vt = ld_in(v, t * a.nv);
    float r = 0.0f, o = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      S[j] *= d;
      r += S[j] * ld_in(k, t * DK + j);
    }
    const float u = b * (vt - group_sum<TPR>(r));
#pragma unroll
    for (int j = 0; j < N; ++j) {
      S[j] += u * ld_in(k, t * DK + j);
      o += S[j] * ld_in(q, t * DK + j);
    }
    o = group_sum<TPR>(o);
    if (c0 == 0 && !__builtin_isfinite(out[t * a.nv])) out[t * a.nv] = o;
  }
  if (a.S_out && seg == a.segs - 1) {
#pragma unroll
    for (int j = 0; j < N; ++j) a.S_out[chain * state + at + j] = S[j];
  }
}

// The running kernel's arguments read anew: what only a rare path needs is not held in
// registers up to it.
__device__ __forceinline__ WalkArgs args_again() {
  unsigned long at = (unsigned long)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(at));
  struct { unsigned w[sizeof(WalkArgs) / 4]; } words;
#pragma unroll
  for (unsigned i = 0; i < sizeof(WalkArgs) / 4; ++i)
    words.w[i] = ((const __attribute__((address_space(4))) unsigned*)at)[i];
  return __builtin_bit_cast(WalkArgs, words);
}

constexpr int threads_of(int nd, bool out) { return 64 * (nd + (out ? out_waves(nd) : kKeyWaves)); }
// Waves a SIMD that registers are held to: two, but where that spills.
template <typename T, int DK, int ND, bool OUT>
constexpr int waves_of() { return OUT && planes<T>() == 3 && DK == 128 ? 1 : 2; }

// OUT: the main walk; else a segment's own write (value rows) and the matrix it multiplies its
// start's rows with (unit rows behind them), 64 of these rows a workgroup.
template <typename T, int DK, int ND, bool OUT>
__global__ __launch_bounds__(threads_of(ND, OUT), (waves_of<T, DK, ND, OUT>())) void walk_kernel(WalkArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  using L = typename std::conditional<OUT, WalkLds<T, DK, ND>, KeyLds<T, DK>>::type;
  constexpr int DZ = 16 * ND;
  L& lds = *reinterpret_cast<L*>(smem);
  const int blocks = OUT ? a.nv / DZ : write_blocks(a.nv + DK);
  const int steps = OUT ? a.segs : a.segs - 1;
  int blk;
  long unit;
  if (!place(blocks, a.chains * steps, blk, unit)) return;
  const long chain = unit / steps;
  const int seg = (int)(unit % steps);
  const long len = a.seqlen, chunks = (len + C - 1) / C, c0 = (long)seg * a.per;
  const int n = (int)(chunks - c0 < a.per ? chunks - c0 : a.per);
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const long left = len - c0 * C;            // tokens from the segment's start on
  const int row0 = blk * DZ;

  if (wave < ND) {
    const int at = row0 + 16 * wave;
    const bool unit_rows = !OUT && at >= a.nv;
    const int row = unit_rows ? at - a.nv : at;
    if (unit_rows && row >= DK) return idle(n);
    Walker<T, DK, typename std::conditional<OUT, RegT, LdsT>::type> w;
    const T* v = static_cast<const T*>(a.v) + (chain * len + c0 * C) * a.nv;
    const uint4* Tp = a.T + (chain * chunks + c0) * kT;
    const long state = (long)a.nv * DK;
    if (unit_rows) w.S.unit(row);
    else if (!OUT) w.S.load(nullptr);
    else if (a.segs > 1) w.S.load(a.starts + (chain * a.segs + seg) * state + (long)row * DK);
    else w.S.load(a.S0 ? a.S0 + chain * state + (long)row * DK : nullptr);
    if constexpr (OUT) w.t.load(Tp);
    // (unit rows have no v: a window of no rows reads 0)
    auto load_v = [&](int c) {
      w.load_v(v + (long)c * C * a.nv, unit_rows ? 0 : left - (long)c * C, a.nv, row);
    };
    load_v(0);
    for (int c = 0; c < n; ++c) {
      __syncthreads();
      if (c == 0) w.load_k(lds.k[0][0]);
      // (what is behind the last chunk is loaded in its own place: no branch holds registers)
      const int next = c + 1 < n ? c + 1 : c;
      if constexpr (!OUT) w.t.p = lds.t[c & 1];
      w.chunk(lds.k[c % L::R][0], lds.gate[c % L::R],
              [&] {
                // (loads come back in order: the one needed first is issued first)
                load_v(next);
                if constexpr (OUT) w.t.load(Tp + (long)next * kT);
              },
              [&] { w.load_k(lds.k[next % L::R][0]); },
              [&](int i, int p, const bf16x8& f) {
                if constexpr (OUT) lds.s[c & 1][wave][i][p][lane] = __builtin_bit_cast(uint4, f);
              },
              [&](const floatx4 (&u)[4]) {
                if constexpr (OUT) {
                  if constexpr (!L::kSplit) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) lds.u[c & 1][wave][i][lane] = __builtin_bit_cast(uint4, u[i]);
                  }
                }
              },
              [&](int i, const floatx4 (&u)[4]) {
                if constexpr (OUT) {
                  if constexpr (L::kSplit) {
                    bf16x8 f[3];
                    frag_pair(u[2 * i], u[2 * i + 1], f);
#pragma unroll
                    for (int p = 0; p < 3; ++p) lds.u[c & 1][wave][3 * i + p][lane] = __builtin_bit_cast(uint4, f[p]);
                  }
                }
              });
    }
    __syncthreads();
    if constexpr (OUT) {
      const bool bad = __any(!w.S.finite());
      if (lane == 0) lds.bad[wave] = bad;
      if (!bad && a.S_out && seg == a.segs - 1) w.S.store(a.S_out + chain * state + (long)row * DK);
      __syncthreads();
    } else if (unit_rows) {
      w.S.store_moves(a.moves + (chain * a.segs + seg) * StateT<DK>::kMove, nullptr, row / 16);
    } else {
      w.S.store(a.starts + (chain * a.segs + seg + 1) * state + (long)row * DK);
    }
  } else {
    if constexpr (OUT) {
      if (wave == ND) outputs<T, DK, ND, 0>(a, lds, chain, c0, n, row0);
      else if (wave == ND + 1) outputs<T, DK, ND, 1>(a, lds, chain, c0, n, row0);
      else if (wave == ND + 2) outputs<T, DK, ND, 2>(a, lds, chain, c0, n, row0);
      else outputs<T, DK, ND, 3>(a, lds, chain, c0, n, row0);
      __syncthreads();
    } else {
      keys_only<T, DK, false>(lds, static_cast<const T*>(a.k) + (chain * len + c0 * C) * DK,
                              a.log_a ? a.log_a + chain * len + c0 * C : nullptr, a.beta + chain * len + c0 * C,
                              a.T + (chain * chunks + c0) * kT, left, n, threadIdx.x - 64 * ND);
    }
  }
  if constexpr (OUT) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < ND; ++i) bad |= lds.bad[i] != 0;
    // (of 16 rows each, so that rows whose result replaced their start stay as they are)
    if (__builtin_expect(bad, 0) && threadIdx.x < 128 * ND && lds.bad[wave / 2]) {
      const WalkArgs again = args_again();
      place(again.nv / DZ, again.chains * again.segs, blk, unit);
      walk_again<T, DK, ND>(again, unit / again.segs, (int)(unit % again.segs), blk * DZ);
    }
  }
}


// ------------------------------------------------------------------- plans

struct Plan {
  int nd, segs, per;
  long chains;
  size_t T_bytes, starts, moves;      // bytes
  size_t bytes() const { return T_bytes + starts + moves; }
  // (a sequence is cut where the launches it takes more have some 256 workgroups)
  bool fit(const DeltaArgs& a) const {
    return solve_fits(chains * (((long)a.seqlen + C - 1) / C)) &&
           fits(a.dv / (16 * nd), chains * segs, threads_of(nd, true));
  }
};
// The segments' first launch and the main walk.
template <typename T, int DK>
void launches(int nd, int nv, Launch& write, Launch& walk) {
  write = {write_blocks(nv + DK), held(sizeof(KeyLds<T, DK>))};
  walk = {nv / (16 * nd), held(nd == 2 ? sizeof(WalkLds<T, DK, 2>) : sizeof(WalkLds<T, DK, 1>))};
}
template <typename T>
void launches(int dk, int nd, int nv, Launch& write, Launch& walk) {
  if (dk == 16) launches<T, 16>(nd, nv, write, walk);
  else if (dk == 32) launches<T, 32>(nd, nv, write, walk);
  else if (dk == 64) launches<T, 64>(nd, nv, write, walk);
  else launches<T, 128>(nd, nv, write, walk);
}
Plan plan_of(const DeltaArgs& a) {
  Plan p;
  p.chains = (long)a.batch * a.heads;
  const long chunks = ((long)a.seqlen + C - 1) / C;
  p.nd = a.dv >= 32 ? 2 : 1;
  if (a.dtype != 0 && a.dk == 128) p.nd = 1;
  Launch write, walk;
  if (a.dtype == 0) launches<uint16_t>(a.dk, p.nd, a.dv, write, walk);
  else launches<float>(a.dk, p.nd, a.dv, write, walk);
  cut(chunks, p.chains, write, 1, walk, a.dk, p.segs, p.per);
  p.T_bytes = (size_t)p.chains * chunks * kT * 16;
  p.starts = p.segs > 1 ? (size_t)p.chains * p.segs * a.dv * a.dk * 4 : 0;
  p.moves = p.segs > 1 ? (size_t)p.chains * p.segs * move_bytes(a.dk) : 0;
  return p;
}

template <typename T, int DK, int ND, bool OUT>
hipError_t go(const WalkArgs& a, hipStream_t stream) {
  constexpr size_t bytes = OUT ? sizeof(WalkLds<T, DK, ND>) : sizeof(KeyLds<T, DK>);
  static_assert(bytes <= 163840, "LDS of a workgroup");
  auto kernel = walk_kernel<T, DK, ND, OUT>;
  const hipError_t e = lds_limit(kernel, bytes);
  if (e != hipSuccess) return e;
  const int blocks = OUT ? a.nv / (16 * ND) : write_blocks(a.nv + DK);
  hipLaunchKernelGGL(kernel, dim3(grid_of(blocks, a.chains * (OUT ? a.segs : a.segs - 1))), dim3(threads_of(ND, OUT)), bytes,
                     stream, a);
  return hipGetLastError();
}

template <typename T>
hipError_t run(const DeltaArgs& a, const Plan& p, hipStream_t stream) {
  char* ws = static_cast<char*>(a.workspace);
  WalkArgs w{a.q, a.k, a.v, a.beta, a.log_a, reinterpret_cast<const uint4*>(ws), a.S0, a.o, a.S_out,
             reinterpret_cast<float*>(ws + p.T_bytes), reinterpret_cast<uint4*>(ws + p.T_bytes + p.starts), p.chains, a.seqlen, a.dv, p.segs, p.per};
  const SolveArgs s{a.k, a.beta, a.log_a, static_cast<uint4*>(a.workspace), nullptr, p.chains, a.seqlen};
  const hipError_t e = launch_solve(s, a.dk, a.dtype, stream);
  if (e != hipSuccess) return e;
  return with_dim(a.dk, [&](auto d) {
    constexpr int DK = decltype(d)::value;
    auto walk = [&](auto nd) {
      constexpr int ND = decltype(nd)::value;
      if (p.segs > 1) {
        hipError_t e = go<T, DK, kWriters, false>(w, stream);
        if (e != hipSuccess) return e;
        const Joins j{{{a.S0, w.starts, w.moves, false}, {}}, p.chains, a.dv, p.segs};
        if ((e = launch_join<DK>(j, 1, stream)) != hipSuccess) return e;
      }
      return go<T, DK, ND, true>(w, stream);
    };
    if constexpr (!(sizeof(T) == 4 && DK == 128)) {
      if (p.nd == 2) return walk(std::integral_constant<int, 2>());
    }
    return walk(std::integral_constant<int, 1>());
  });
}

}  // namespace
}  // namespace delta

size_t delta_workspace_bytes(const DeltaArgs& a) { return delta::plan_of(a).bytes(); }

bool delta_fits(const DeltaArgs& a) { return delta::plan_of(a).fit(a); }

hipError_t launch_delta(const DeltaArgs& a, hipStream_t stream) {
  (void)hipGetLastError();
  const delta::Plan p = delta::plan_of(a);
  return a.dtype == 0 ? delta::run<uint16_t>(a, p, stream) : delta::run<float>(a, p, stream);
}

}  // namespace falcon
