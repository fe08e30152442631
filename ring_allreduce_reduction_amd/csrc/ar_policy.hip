// ar_policy.hip -- the clipped policy loss with a KL term over every rank's
// tokens, and its gradient.
//
// A token with log-probability l under the policy, o under the one that
// sampled it, f under a reference, advantage A and weight w:
//   r = exp(l - o),  loss = -min(A r, A clamp(r, 1 - low, 1 + high)),
//   kl = exp(f - l) - (f - l) - 1,
//   L = sum w (loss + beta kl) / W,  W = the sum of all weights or given,
//   dL/dl = w / W (-A r [not clipped] + beta (1 - exp(f - l))).
// The mean is over all ranks, so the gradient's factor is a sum over every
// token: the first pass leaves the sums and the gradients short of that factor
// and of their weights, the second multiplies them by both (reading the weights
// again: 8 x 262144 tokens 16.5-16.9 us, 16.0-16.4 where the first pass applied
// them in 32 bits, which weights far from 1 leave).  Whether a ratio passes a
// bound is decided by differences in 64 bits against the bounds' logarithms, since
// these are numbers that may nearly agree; the sums are in 64 bits; what lies
// between is formed in 32, kl by its series where it is a difference of nearly
// equal numbers.
//
// Times in comments are of calls in a replayed graph; a call from the host takes
// up to 1.6 us longer where it is short.
#include <cmath>
#include <new>
#include <vector>

#include "ar_rows.h"

namespace ar {
namespace {

constexpr int kPolBlock = 256;
constexpr int kPolSums = 4;            // weights, weighted loss, kl, clipped tokens
// Workgroups, and partial sums, of a launch at most, and where they do with a
// vector a thread: 8 x 262144 tokens 16.5 us with 2 a CU, 20.4 with 1, 17.0 with
// 4, 19.6 with 8, whose sums cost as much as their tokens; 8 x 75000 8.7 with 4 a
// CU and 9.4 with 2, x 100000 10.0 and 10.2, without weights 8.7 and 8.1.  Two
// vectors a thread in flight in the first pass cost a tenth.
constexpr int kPolGrid = 2 * kOpsCUs, kPolOnce = 4 * kOpsCUs;
constexpr int kPolVec = 4;             // tokens of a thread at a time
constexpr int kPolFewBlock = 1024;
constexpr int kPolFewEach = 5;
// Tokens of one workgroup's launch: its wavefronts' parts of 64, less what the
// ranks leave of their last ones.  8 x 64 tokens 3.7 us (6.0 in two launches), x
// 256 4.8 (5.9), x 512 6.3 (6.1); 6000 of one rank 7.5 (5.9).
constexpr int kPolFew = kPolFewBlock * kPolFewEach - kOpRanks * kWave;

// Ranks of a launch at most.  Up to kOpRanks of them travel in arguments of
// that size, which take the host less time to hand over (1250 tokens of 4 ranks,
// calls from the host, 4.8 us, 5.2 with twice the size; 20 ranks through the
// binding 6.5, 18 in two launches and a third).
constexpr int kPolRanks = 2 * kOpRanks;

struct PolCall {
  int nranks;
  int partials;                        // of all launches
  double* partial;                     // kPolSums rows of `partials`; the first pass: from this launch's first
  float* stats;                        // where the launch writes them, or null
  double klCoef, denominator, gradScale;
  double over;                         // what the sums are divided by, where the host knows it; else 0
  double logLow, logHigh;              // log(1 - low), log(1 + high)
  float low, high;                     // 1 - low, 1 + high
  float klGrad;                        // klCoef in 32 bits, 0 only where it is
  bool hasRef;
};

// What the second pass needs, and what the first needs besides.
template <int RANKS>
struct PolGradArgs : PolCall {
  float* dlogp[RANKS];                 // null pointers: not wanted
  const float* weight[RANKS];          // null pointers: 1
  int start[RANKS + 1];                // rank r has tokens [start[r], start[r + 1]) of the launch
  int blockStart[RANKS + 1];           // and workgroups [blockStart[r], blockStart[r + 1])
};

template <int RANKS>
struct PolArgs : PolGradArgs<RANKS> {
  const float* logp[RANKS];
  const float* old[RANKS];
  const float* ref[RANKS];             // null pointers: no KL term
  const float* advantage[RANKS];

  // Those of another size, whose ranks fit.
  template <int OTHER>
  static PolArgs of(const PolArgs<OTHER>& a) {
    PolArgs to{};
    (PolCall&)to = a;
    for (int r = 0; r < a.nranks; ++r) {
      to.dlogp[r] = a.dlogp[r];
      to.logp[r] = a.logp[r];
      to.old[r] = a.old[r];
      to.ref[r] = a.ref[r];
      to.advantage[r] = a.advantage[r];
      to.weight[r] = a.weight[r];
    }
    for (int r = 0; r <= a.nranks; ++r) {
      to.start[r] = a.start[r];
      to.blockStart[r] = a.blockStart[r];
    }
    return to;
  }
};

typedef int Halves __attribute__((ext_vector_type(2)));   // of 64 bits

struct Token {
  float loss, kl, dlogp;
  bool clipped;
};

__device__ __forceinline__ float expFast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f); }

// exp(d) - 1 and exp(d) - 1 - d, below |d| = 1 from the exponential's series
// through d^12 (what is left out is 2^-31 of the result): there they are
// differences of nearly equal numbers.  An infinite d counts as the largest
// number: its exponential outgrows it.
__device__ __forceinline__ float2 expLess(float d) {
  d = __builtin_elementwise_minimum(d, 0x1.fffffep127f);   // NaN stays
  constexpr double kOver[13] = {0, 0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040, 1.0 / 40320,
                                1.0 / 362880, 1.0 / 3628800, 1.0 / 39916800, 1.0 / 479001600};
  float s = (float)kOver[12];
#pragma unroll
  for (int n = 11; n >= 2; --n) s = fmaf(s, d, (float)kOver[n]);
  const float near = d * d * s, e = expFast(d) - 1.0f;
  const bool small = fabsf(d) < 1.0f;
  return make_float2(small ? near + d : e, small ? near : e - d);
}

__device__ __forceinline__ Token tokenOf(const PolCall& a, float logp, float old, float advantage, bool hasRef,
                                         float ref) {
  Token t;
  const double change = (double)logp - (double)old;
  const bool up = advantage > 0.0f && change > a.logHigh, down = advantage < 0.0f && change < a.logLow;
  // An advantage of 0 takes no part, not of an infinite ratio either.  Without a
  // branch: 8 x 262144 tokens 16.4 us, 19.0 with one.
  const float e = expFast((float)change);
  const bool idle = (advantage == 0.0f) & (e == INFINITY);
  const float ratio = idle ? 0.0f : e;
  t.clipped = up || down;
  t.loss = -advantage * (up ? a.high : down ? a.low : ratio);
  t.dlogp = t.clipped ? 0.0f : -advantage * ratio;
  t.kl = 0.0f;
  if (hasRef) {
    const float2 less = expLess((float)((double)ref - (double)logp));
    t.kl = less.y;
    // of coefficient 0 it is only reported, and may be infinite
    if (a.klGrad != 0.0f) t.dlogp -= a.klGrad * less.x;
  }
  return t;
}

// What lane permutation CTRL brings.
template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
  const auto b = __builtin_bit_cast(Halves, v);
  return __builtin_bit_cast(double, Halves{__builtin_amdgcn_update_dpp(0, b[0], CTRL, 0xf, 0xf, true),
                                           __builtin_amdgcn_update_dpp(0, b[1], CTRL, 0xf, 0xf, true)});
}

// v plus that of the lane 16 (ROWS) or 32 further on, modulo twice as much.
template <bool ROWS>
__device__ __forceinline__ double addHalves(double v) {
  const auto b = __builtin_bit_cast(Halves, v);
  const auto swap = [](int h) {
    return ROWS ? __builtin_amdgcn_permlane16_swap(h, h, false, false)
                : __builtin_amdgcn_permlane32_swap(h, h, false, false);
  };
  const auto low = swap(b[0]), high = swap(b[1]);
  return __builtin_bit_cast(double, Halves{(int)low[0], (int)high[0]}) +
         __builtin_bit_cast(double, Halves{(int)low[1], (int)high[1]});
}

// Sum over those of LANES lanes side by side whose index agrees modulo 4; each
// receives its own, the same in all of them.
template <int LANES>
__device__ __forceinline__ double sumFourths(double v) {
  static_assert(LANES == 16 || LANES == 64, "a row or a wavefront");
  v += dpp64<0x128>(v);   // row_ror 8
  v += dpp64<0x124>(v);   // row_ror 4
  return LANES == 16 ? v : addHalves<false>(addHalves<true>(v));
}

// Sum over quads; each of their lanes receives it.
__device__ __forceinline__ double sumQuad(double v) {
  v += dpp64<0xb1>(v);          // quad_perm 1,0,3,2
  return v + dpp64<0x4e>(v);    // quad_perm 2,3,0,1
}

// Sum over a workgroup of four wavefronts; every thread receives it.
__device__ __forceinline__ double blockSum64(double s, double (&lds)[4]) {
  s = sumFourths<kWave>(sumQuad(s));
  if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = s;
  __syncthreads();
  return sumQuad(lds[threadIdx.x % 4]);
}

// Four sums over a workgroup of 4 or 16 wavefronts; thread i receives number
// i % 4.  Neighbours hand each other what they do not keep, so that after two
// steps a lane holds one of the four; the wavefronts' are read one a lane.
template <int BLOCK>
__device__ __forceinline__ double blockSums(const double (&s)[kPolSums], double (&lds)[BLOCK / kWave * kPolSums]) {
  static_assert(kPolSums == 4, "one a lane of a quad");
  const bool odd = threadIdx.x & 1, second = threadIdx.x & 2;
  const double a = (odd ? s[1] : s[0]) + dpp64<0xb1>(odd ? s[0] : s[1]);
  const double b = (odd ? s[3] : s[2]) + dpp64<0xb1>(odd ? s[2] : s[3]);
  const double v = sumFourths<kWave>((second ? b : a) + dpp64<0x4e>(second ? a : b));
  const int lane = (int)threadIdx.x % kWave;
  if (lane < kPolSums) lds[threadIdx.x / kWave * kPolSums + lane] = v;
  __syncthreads();
  constexpr int ALL = BLOCK / kWave * kPolSums;
  return sumFourths<ALL>(lds[threadIdx.x % ALL]);
}

// What lane `lane` of the wavefront holds.
__device__ __forceinline__ double laneOf(double v, int lane) {
  const auto b = __builtin_bit_cast(Halves, v);
  return __builtin_bit_cast(double, Halves{__builtin_amdgcn_readlane(b[0], lane), __builtin_amdgcn_readlane(b[1], lane)});
}

// Adds a token up and returns its gradient short of its weight and the common
// factor.  One of weight 0 is left out, whatever its other values are.
__device__ __forceinline__ float addToken(const PolCall& a, float logp, float old, float advantage, bool hasRef,
                                          float ref, float weight, double (&s)[kPolSums]) {
  const Token t = tokenOf(a, logp, old, advantage, hasRef, ref);
  const bool counts = weight != 0.0f;
  const double w = weight;
  s[0] += w;
  s[1] = fma(w, (double)(counts ? t.loss : 0.0f), s[1]);
  s[2] = fma(w, (double)(counts ? t.kl : 0.0f), s[2]);
  s[3] += t.clipped ? w : 0.0;
  return counts ? t.dlogp : 0.0f;
}

__device__ __forceinline__ double partOf(const PolCall& a, double weights) {
  const double over = a.denominator > 0.0 ? a.denominator : weights;
  return over != 0.0 ? 1.0 / over : 0.0;
}

// The gradients' common factor, held at the largest number, so that it leaves a
// gradient of 0 at 0 (and makes any other infinite).
__device__ __forceinline__ double factorOf(double f) {
  return fabs(f) == INFINITY ? copysign(0x1.fffffffffffffp1023, f) : f;
}

// Called by the workgroup's threads with what blockSums gave them.
__device__ __forceinline__ void putStats(const PolCall& a, double sums) {
  const double weights = laneOf(sums, 0), loss = laneOf(sums, 1), klSum = laneOf(sums, 2), clipped = laneOf(sums, 3);
  if (threadIdx.x > 0) return;
  const double part = partOf(a, weights), policy = loss * part, kl = klSum * part;
  a.stats[0] = (float)(a.klCoef != 0.0 ? policy + a.klCoef * kl : policy);
  a.stats[1] = (float)policy;
  a.stats[2] = (float)kl;
  a.stats[3] = (float)(clipped * part);
  a.stats[4] = (float)weights;
}

// A gradient and what it was short of, in 64 bits, since all weights and their
// sum may be far from 1; 0 where nothing counts, whatever the gradient is.
__device__ __forceinline__ float timesFactor(float d, float weight, double factor) {
  return factor != 0.0 ? (float)((double)d * (double)weight * factor) : 0.0f;
}

// A workgroup's rank, and a thread's share of that rank's tokens: every
// step-th vector from the first, and one of the few tokens behind the last.
struct PolPlace {
  int rank, count, whole;
  int64_t first, step;
};

template <int RANKS>
__device__ __forceinline__ PolPlace polPlace(const PolGradArgs<RANKS>& a) {
  PolPlace p;
  p.rank = 0;
  while ((int)blockIdx.x >= a.blockStart[p.rank + 1]) ++p.rank;
  const int block = (int)blockIdx.x - a.blockStart[p.rank];
  p.count = a.start[p.rank + 1] - a.start[p.rank];
  p.whole = p.count / kPolVec * kPolVec;
  p.first = ((int64_t)block * kPolBlock + threadIdx.x) * kPolVec;
  p.step = (int64_t)(a.blockStart[p.rank + 1] - a.blockStart[p.rank]) * kPolBlock * kPolVec;
  return p;
}

// Calls f(first token) for a thread's vectors but the first `done`, then g(token) for its part of
// the rest, which the rank's first workgroup takes.
template <typename F, typename G>
__device__ __forceinline__ void forTokens(const PolPlace& p, int done, F f, G g) {
  int64_t i = p.first + done * p.step;
  for (; i < p.whole; i += p.step) f(i);
  i = p.whole + p.first / kPolVec;
  if (i < p.count) g(i);
}

template <int RANKS>
__global__ void __launch_bounds__(kPolBlock) policySums(const PolArgs<RANKS> a) {
  __shared__ double lds[kPolBlock / kWave * kPolSums];
  const PolPlace at = polPlace<RANKS>(a);
  const float *logp = a.logp[at.rank], *old = a.old[at.rank], *ref = a.ref[at.rank];
  const float *advantage = a.advantage[at.rank], *weight = a.weight[at.rank];
  float* dlogp = a.dlogp[at.rank];
  double s[kPolSums] = {0.0, 0.0, 0.0, 0.0};
  typedef FloatVec<kPolVec> Vec;
  const bool known = a.over > 0.0;
  const double factor = known ? factorOf(a.gradScale / a.over) : 1.0;
  forTokens(
      at, 0,
      [&](int64_t i) {
        const Vec l = loadVec<float, kPolVec>(logp + i), o = loadVec<float, kPolVec>(old + i);
        const Vec v = loadVec<float, kPolVec>(advantage + i);
        const Vec f = ref ? loadVec<float, kPolVec>(ref + i) : (Vec)0.0f;
        const Vec w = weight ? loadVec<float, kPolVec>(weight + i) : (Vec)1.0f;
        Vec d;
#pragma unroll
        for (int e = 0; e < kPolVec; ++e) d[e] = addToken(a, l[e], o[e], v[e], ref != nullptr, f[e], w[e], s);
        if (known)
#pragma unroll
          for (int e = 0; e < kPolVec; ++e) d[e] = timesFactor(d[e], w[e], factor);
        if (dlogp) storeVec<float, kPolVec>(dlogp + i, d);
      },
      [&](int64_t i) {
        const float w = weight ? weight[i] : 1.0f;
        const float d = addToken(a, logp[i], old[i], advantage[i], ref != nullptr, ref ? ref[i] : 0.0f, w, s);
        if (dlogp) dlogp[i] = known ? timesFactor(d, w, factor) : d;
      });
  const double sums = blockSums<kPolBlock>(s, lds);
  if (threadIdx.x < kPolSums) a.partial[(size_t)threadIdx.x * a.partials + blockIdx.x] = sums;
}

// The sums of the first pass in one order for every workgroup: what each
// gradient's factor needs of them, and, where the launch writes the stats, all
// of them in its last workgroup, which has no tokens.
template <int RANKS>
__global__ void __launch_bounds__(kPolBlock) policyGrad(const PolGradArgs<RANKS> a) {
  typedef FloatVec<kPolVec> Vec;
  if (a.stats && blockIdx.x == gridDim.x - 1) {
    __shared__ double lds[kPolBlock / kWave * kPolSums];
    double s[kPolSums] = {0.0, 0.0, 0.0, 0.0};
    for (int i = threadIdx.x; i < a.partials; i += kPolBlock)
#pragma unroll
      for (int k = 0; k < kPolSums; ++k) s[k] += a.partial[(size_t)k * a.partials + i];
    putStats(a, blockSums<kPolBlock>(s, lds));
    return;
  }
  __shared__ double lds[kPolBlock / kWave];
  const PolPlace at = polPlace(a);
  float* dlogp = a.dlogp[at.rank];
  const float* weight = a.weight[at.rank];   // there are some, or their sum was known before
  // a thread's first vector is on its way while the sums are joined (8 x 262144
  // tokens 16.5 us, with its first four 16.5, eight 16.5; x 1 M 49.6, 49.7, 50.4; x
  // 12500 6.3, 6.5, 6.6)
  const bool any = at.first < at.whole;
  Vec ahead = (Vec)0.0f, weightAhead = (Vec)0.0f;
  if (any) {
    ahead = loadVec<float, kPolVec>(dlogp + at.first);
    weightAhead = loadVec<float, kPolVec>(weight + at.first);
  }
  double weights = 0.0;
  for (int i = threadIdx.x; i < a.partials; i += kPolBlock) weights += a.partial[i];
  weights = blockSum64(weights, lds);
  const double factor = factorOf(a.gradScale * partOf(a, weights));
  const auto put = [&](int64_t i, Vec d, const Vec& w) {
#pragma unroll
    for (int e = 0; e < kPolVec; ++e) d[e] = timesFactor(d[e], w[e], factor);
    storeVec<float, kPolVec>(dlogp + i, d);
  };
  if (any) put(at.first, ahead, weightAhead);
  forTokens(
      at, 1, [&](int64_t i) { put(i, loadVec<float, kPolVec>(dlogp + i), loadVec<float, kPolVec>(weight + i)); },
      [&](int64_t i) { dlogp[i] = timesFactor(dlogp[i], weight[i], factor); });
}

// Few tokens: one workgroup, one launch, the gradients kept in registers until
// their factor is known.  A wavefront takes 64 tokens of a rank at a time.
template <int RANKS>
__global__ void __launch_bounds__(kPolFewBlock) policyFew(const PolArgs<RANKS> a) {
  constexpr int WAVES = kPolFewBlock / kWave;
  __shared__ double lds[WAVES * kPolSums];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave), lane = (int)threadIdx.x % kWave;
  // all of a thread's tokens are on their way before the first is looked at
  float logp[kPolFewEach], old[kPolFewEach], advantage[kPolFewEach], ref[kPolFewEach], weight[kPolFewEach];
  float *dlogp[kPolFewEach], d[kPolFewEach];
  bool any[kPolFewEach];
  const bool hasRef = a.hasRef;
  int r = 0;
#pragma unroll
  for (int k = 0; k < kPolFewEach; ++k) {
    const int piece = wave + k * WAVES;
    any[k] = piece < a.blockStart[a.nranks];
    if (!any[k]) continue;
    while (piece >= a.blockStart[r + 1]) ++r;
    const int i = (piece - a.blockStart[r]) * kWave + lane;
    any[k] = i < a.start[r + 1] - a.start[r];
    dlogp[k] = a.dlogp[r] ? a.dlogp[r] + i : nullptr;
    if (!any[k]) continue;
    logp[k] = a.logp[r][i];
    old[k] = a.old[r][i];
    advantage[k] = a.advantage[r][i];
    ref[k] = hasRef ? a.ref[r][i] : 0.0f;
    weight[k] = a.weight[r] ? a.weight[r][i] : 1.0f;
  }
  double s[kPolSums] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
  for (int k = 0; k < kPolFewEach; ++k)
    if (any[k]) d[k] = addToken(a, logp[k], old[k], advantage[k], hasRef, ref[k], weight[k], s);
  const double sums = blockSums<kPolFewBlock>(s, lds);
  putStats(a, sums);
  const double factor = factorOf(a.gradScale * partOf(a, laneOf(sums, 0)));
#pragma unroll
  for (int k = 0; k < kPolFewEach; ++k)
    if (any[k] && dlogp[k]) *dlogp[k] = timesFactor(d[k], weight[k], factor);
}

// Shares a launch's tokens out among its workgroups, one partial sum each, or,
// `few`, among a workgroup's wavefronts; returns their number.
int cutTokens(const size_t* tokens, int ranks, bool few, int* start, int* blockStart) {
  const int each = few ? kWave : kPolBlock * kPolVec;
  start[0] = blockStart[0] = 0;
  for (int r = 0; r < ranks; ++r) start[r + 1] = start[r] + (int)tokens[r];
  const int most = wholeGroups(start, ranks, each) <= kPolOnce ? kPolOnce : kPolGrid;
  return giveOut(start, ranks, each, each, most, blockStart);
}

// Of more than kOpRanks ranks less, since each may leave 63 threads of a part.
bool polFew(const Shape& s, int nranks) {
  if (s.total == 0) return true;
  return nranks <= kPolRanks && s.total <= kPolFew - (nranks > kOpRanks ? (kPolRanks - kOpRanks) * kWave : 0);
}

int polLaunches(int nranks) { return (nranks + kPolRanks - 1) / kPolRanks; }

arResult_t polWorkspace(const size_t* tokens, int nranks, size_t* bytes) {
  Shape s;
  if (bytes == nullptr || !rowsOk(tokens, nranks, &s)) return arInvalidArgument;
  size_t partials = 0;
  int start[kPolRanks + 1], blockStart[kPolRanks + 1];
  if (!polFew(s, nranks))
    for (int first = 0; first < nranks; first += kPolRanks)
      partials += (size_t)cutTokens(tokens + first, nranks - first < kPolRanks ? nranks - first : kPolRanks,
                                    false, start, blockStart);
  *bytes = partials * kPolSums * sizeof(double);
  return arSuccess;
}

void fillTokens(PolArgs<kPolRanks>* a, const float* const* logp, const float* const* old, const float* const* ref,
                const float* const* advantage, const float* const* weight, float* const* dlogp, const size_t* tokens,
                int nranks, int first, bool few) {
  a->nranks = nranks - first < kPolRanks ? nranks - first : kPolRanks;
  cutTokens(tokens + first, a->nranks, few, a->start, a->blockStart);
  for (int r = 0; r < a->nranks; ++r) {
    const int k = first + r;
    const bool any = tokens[k] > 0;
    a->logp[r] = any ? logp[k] : nullptr;
    a->old[r] = any ? old[k] : nullptr;
    a->ref[r] = any && ref ? ref[k] : nullptr;
    a->advantage[r] = any ? advantage[k] : nullptr;
    a->weight[r] = any && weight ? weight[k] : nullptr;
    a->dlogp[r] = any && dlogp ? dlogp[k] : nullptr;
  }
}

// With arguments of the size that the ranks need.
template <typename A, typename B>
bool polLaunch(void (*kernel)(A), void (*larger)(B), int grid, int block, const PolArgs<kPolRanks>& a, hipStream_t st) {
  if (a.nranks > kOpRanks) return launchKernel<B>(larger, dim3(grid), dim3(block), a, st) == hipSuccess;
  return launchKernel<A>(kernel, dim3(grid), dim3(block), PolArgs<kOpRanks>::of(a), st) == hipSuccess;
}

arResult_t policyLoss(const float* const* logp, const float* const* old, const float* const* ref,
                      const float* const* advantage, const float* const* weight, float* const* dlogp,
                      const size_t* tokens, int nranks, double clipLow, double clipHigh, double klCoef,
                      double denominator, double gradScale, float* stats, void* workspace, size_t workspaceGiven,
                      hipStream_t st) {
  Shape s;
  if (!rowsOk(tokens, nranks, &s) || !aligned(stats, 4)) return arInvalidArgument;
  if (!(clipLow >= 0.0 && clipLow <= 1.0) || !(clipHigh >= 0.0)) return arInvalidArgument;
  if (!(klCoef >= 0.0 && klCoef <= 0x1.fffffep127) || !std::isfinite(gradScale)) return arInvalidArgument;
  if (denominator != 0.0 && !(denominator > 0.0 && std::isnormal(denominator))) return arInvalidArgument;
  if (klCoef != 0.0 && ref == nullptr) return arInvalidArgument;
  if (groupOpen()) return arInvalidUsage;
  if (s.total > 0 && (logp == nullptr || old == nullptr || advantage == nullptr)) return arInvalidArgument;
  std::vector<Extent> v;
  v.reserve((size_t)nranks * 6 + 2);
  bool ok = addFlat(v, stats, 5, 4, true);
  for (int r = 0; r < nranks; ++r) {
    const size_t n = tokens[r];
    if (n == 0) continue;
    ok = ok && addRows(v, logp[r], 1, n, n, 4, false, r) && addFlat(v, old[r], n, 4, false) &&
         addFlat(v, advantage[r], n, 4, false);
    if (ref != nullptr) ok = ok && addFlat(v, ref[r], n, 4, false);
    if (weight != nullptr) ok = ok && addFlat(v, weight[r], n, 4, false);
    if (dlogp != nullptr) ok = ok && addRows(v, dlogp[r], 1, n, n, 4, true, r);
  }
  if (!ok) return arInvalidArgument;
  const bool few = polFew(s, nranks);
  if (!few) {
    size_t need = 0;
    const arResult_t r = polWorkspace(tokens, nranks, &need);
    if (r != arSuccess) return r;
    if (workspace == nullptr || (uintptr_t)workspace % 16 != 0 || workspaceGiven < need) return arInvalidArgument;
    v.push_back(Extent{(uintptr_t)workspace, need, 1, need, true, -1});
  }
  if (outputsOverlap(v)) return arInvalidArgument;
  PolArgs<kPolRanks> a{};
  a.hasRef = ref != nullptr;
  a.low = (float)(1.0 - clipLow);
  a.high = (float)(1.0 + clipHigh);
  a.logLow = std::log1p(-clipLow);
  a.logHigh = std::log1p(clipHigh);
  a.klCoef = klCoef;
  a.klGrad = klCoef > 0.0 && klCoef < 0x1p-149 ? 0x1p-149f : (float)klCoef;
  a.denominator = denominator;
  a.gradScale = gradScale;
  a.over = denominator > 0.0 ? denominator : weight == nullptr ? (double)s.total : 0.0;
  if (few) {
    fillTokens(&a, logp, old, ref, advantage, weight, dlogp, tokens, nranks, 0, true);
    a.stats = stats;
    return polLaunch(policyFew<kOpRanks>, policyFew<kPolRanks>, 1, kPolFewBlock, a, st) ? arSuccess : arHipError;
  }
  for (int l = 0; l < polLaunches(nranks); ++l) {
    fillTokens(&a, logp, old, ref, advantage, weight, dlogp, tokens, nranks, l * kPolRanks, false);
    a.partials += a.blockStart[a.nranks];
  }
  int partials = 0;
  for (int l = 0; l < polLaunches(nranks); ++l) {
    fillTokens(&a, logp, old, ref, advantage, weight, dlogp, tokens, nranks, l * kPolRanks, false);
    const int grid = a.blockStart[a.nranks];
    if (grid == 0) continue;
    a.partial = (double*)workspace + partials;
    if (!polLaunch(policySums<kOpRanks>, policySums<kPolRanks>, grid, kPolBlock, a, st)) return arHipError;
    partials += grid;
  }
  a.partial = (double*)workspace;
  // with a factor known beforehand the gradients are whole, and the stats are
  // left (8 x 262144 tokens without weights 14.5 us, with them 18.5)
  float* const* unscaled = a.over > 0.0 ? nullptr : dlogp;
  for (int l = 0; l < polLaunches(nranks); ++l) {
    fillTokens(&a, logp, old, ref, advantage, weight, unscaled, tokens, nranks, l * kPolRanks, false);
    a.stats = l == 0 ? stats : nullptr;
    const int grid = (unscaled != nullptr ? a.blockStart[a.nranks] : 0) + (l == 0 ? 1 : 0);
    if (grid == 0) continue;
    if (!polLaunch(policyGrad<kOpRanks>, policyGrad<kPolRanks>, grid, kPolBlock, a, st)) return arHipError;
  }
  return arSuccess;
}

}  // namespace
}  // namespace ar

extern "C" arResult_t arPolicyLossWorkspace(const size_t* tokens, int nranks, size_t* bytes) {
  return ar::polWorkspace(tokens, nranks, bytes);
}

extern "C" arResult_t arPolicyLoss(const float* const* logp, const float* const* old, const float* const* ref,
                                   const float* const* advantage, const float* const* weight, float* const* dlogp,
                                   const size_t* tokens, int nranks, double clipLow, double clipHigh, double klCoef,
                                   double denominator, double gradScale, float* stats, void* workspace,
                                   size_t workspaceBytes, void* stream) {
  ApiRange range("arPolicyLoss");
  try {
    return ar::noteGroupError(ar::policyLoss(logp, old, ref, advantage, weight, dlogp, tokens, nranks, clipLow,
                                             clipHigh, klCoef, denominator, gradScale, stats, workspace,
                                             workspaceBytes, (hipStream_t)stream));
  } catch (const std::bad_alloc&) {
    return ar::noteGroupError(arSystemError);
  }
}
