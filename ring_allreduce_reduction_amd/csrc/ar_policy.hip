// ar_policy.hip -- the clipped policy loss with a KL term over every rank's
// tokens, and its gradient.
//
// A token with log-probability l under the policy, o under the one that
// sampled it, f under a reference, advantage A and weight w:
//   r = exp(l - o),  loss = -min(A r, A clamp(r, 1 - low, 1 + high)),
//   kl = exp(f - l) - (f - l) - 1,
//   L = sum w (loss + beta kl) / W,  W = the sum of all weights or given,
//   dL/dl = w / W (-A r [not clipped] + beta (1 - exp(f - l))).
// The mean is over all ranks, so the gradient needs a sum of every token
// first: two passes, the second from the caches.  A token's terms are formed
// in 64 bits: whether its ratio passes a bound is a comparison of numbers that
// nearly agree, kl is a difference of nearly equal numbers, and the sums may be
// long.
#include <cmath>
#include <new>
#include <vector>

#include "ar_rows.h"

namespace ar {
namespace {

constexpr int kPolBlock = 256;
constexpr int kPolSums = 4;            // weighted loss, kl, clipped tokens, weights
constexpr int kPolGrid = 2 * kOpsCUs;  // workgroups, and partial sums, of a launch at most
constexpr int kPolFew = 4096;          // tokens of one workgroup's launch
constexpr int kPolFewBlock = 1024;

struct PolArgs {
  const float* logp[kOpRanks];
  const float* old[kOpRanks];
  const float* ref[kOpRanks];          // null pointers: no KL term
  const float* advantage[kOpRanks];
  const float* weight[kOpRanks];       // null pointers: 1
  float* dlogp[kOpRanks];              // null pointers: not wanted
  int start[kOpRanks + 1];             // rank r has tokens [start[r], start[r + 1]) of the launch
  int blockStart[kOpRanks + 1];        // and workgroups [blockStart[r], blockStart[r + 1])
  int nranks;
  int partials;                        // of all launches
  double* partial;                     // kPolSums rows of `partials`; the first pass: from this launch's first
  float* stats;                        // where the launch writes them, or null
  double logLow, logHigh;              // log(1 - low), log(1 + high)
  double low, high;                    // 1 - low, 1 + high
  double klCoef, denominator, gradScale;
};

struct Token {
  double loss, kl, clipped, dlogp;
};

__device__ __forceinline__ Token tokenOf(const PolArgs& a, float logp, float old, float advantage, bool hasRef,
                                         float ref) {
  Token t;
  const double change = (double)logp - (double)old, adv = advantage;
  const bool up = adv > 0.0 && change > a.logHigh, down = adv < 0.0 && change < a.logLow;
  const double ratio = exp(change);
  t.clipped = up || down ? 1.0 : 0.0;
  t.loss = -adv * (up ? a.high : down ? a.low : ratio);
  t.dlogp = up || down ? 0.0 : -adv * ratio;
  t.kl = 0.0;
  if (hasRef) {
    const double d = (double)ref - (double)logp, e = expm1(d);
    t.kl = e - d;
    t.dlogp -= a.klCoef * e;
  }
  return t;
}

__device__ __forceinline__ double waveSum64(double v) {
#pragma unroll
  for (int m = 1; m < kWave; m *= 2) v += __shfl_xor(v, m);
  return v;
}

// Sums of four over a workgroup; every thread receives them.
template <int BLOCK>
__device__ __forceinline__ void blockSums(double (&s)[kPolSums], double (*lds)[kPolSums]) {
#pragma unroll
  for (int k = 0; k < kPolSums; ++k) s[k] = waveSum64(s[k]);
  if (threadIdx.x % kWave == 0)
#pragma unroll
    for (int k = 0; k < kPolSums; ++k) lds[threadIdx.x / kWave][k] = s[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPolSums; ++k) {
    s[k] = lds[0][k];
    for (int w = 1; w < BLOCK / kWave; ++w) s[k] += lds[w][k];
  }
}

__device__ __forceinline__ void addToken(const PolArgs& a, int r, int i, double (&s)[kPolSums]) {
  const double w = a.weight[r] ? (double)a.weight[r][i] : 1.0;
  if (w == 0.0) return;
  const Token t = tokenOf(a, a.logp[r][i], a.old[r][i], a.advantage[r][i], a.ref[r] != nullptr,
                          a.ref[r] ? a.ref[r][i] : 0.0f);
  s[0] += w * t.loss;
  s[1] += w * t.kl;
  s[2] += w * t.clipped;
  s[3] += w;
}

__device__ __forceinline__ double partOf(const PolArgs& a, double weights) {
  const double over = a.denominator > 0.0 ? a.denominator : weights;
  return over != 0.0 ? 1.0 / over : 0.0;
}

__device__ __forceinline__ void putStats(const PolArgs& a, const double (&s)[kPolSums]) {
  const double part = partOf(a, s[3]), policy = s[0] * part, kl = s[1] * part;
  a.stats[0] = (float)(policy + a.klCoef * kl);
  a.stats[1] = (float)policy;
  a.stats[2] = (float)kl;
  a.stats[3] = (float)(s[2] * part);
  a.stats[4] = (float)s[3];
}

__device__ __forceinline__ void putGrad(const PolArgs& a, int r, int i, double factor) {
  const double w = a.weight[r] ? (double)a.weight[r][i] : 1.0;
  float d = 0.0f;
  if (w != 0.0 && factor != 0.0) {
    const Token t = tokenOf(a, a.logp[r][i], a.old[r][i], a.advantage[r][i], a.ref[r] != nullptr,
                            a.ref[r] ? a.ref[r][i] : 0.0f);
    d = (float)(factor * w * t.dlogp);
  }
  a.dlogp[r][i] = d;
}

// A workgroup's rank, and its share of that rank's tokens: every step-th from
// the first.
struct PolPlace {
  int rank, first, step, count;
};

__device__ __forceinline__ PolPlace polPlace(const PolArgs& a) {
  PolPlace p;
  p.rank = 0;
  while ((int)blockIdx.x >= a.blockStart[p.rank + 1]) ++p.rank;
  p.first = ((int)blockIdx.x - a.blockStart[p.rank]) * kPolBlock + (int)threadIdx.x;
  p.step = (a.blockStart[p.rank + 1] - a.blockStart[p.rank]) * kPolBlock;
  p.count = a.start[p.rank + 1] - a.start[p.rank];
  return p;
}

__global__ void __launch_bounds__(kPolBlock) policySums(const PolArgs a) {
  __shared__ double lds[kPolBlock / kWave][kPolSums];
  const PolPlace at = polPlace(a);
  double s[kPolSums] = {0.0, 0.0, 0.0, 0.0};
  for (int64_t i = at.first; i < at.count; i += at.step) addToken(a, at.rank, (int)i, s);
  blockSums<kPolBlock>(s, lds);
  if (threadIdx.x == 0)
#pragma unroll
    for (int k = 0; k < kPolSums; ++k) a.partial[(size_t)k * a.partials + blockIdx.x] = s[k];
}

__global__ void __launch_bounds__(kPolBlock) policyGrad(const PolArgs a) {
  __shared__ double lds[kPolBlock / kWave][kPolSums];
  double s[kPolSums] = {0.0, 0.0, 0.0, 0.0};
  for (int i = threadIdx.x; i < a.partials; i += kPolBlock)
#pragma unroll
    for (int k = 0; k < kPolSums; ++k) s[k] += a.partial[(size_t)k * a.partials + i];
  blockSums<kPolBlock>(s, lds);
  if (a.stats && blockIdx.x == 0 && threadIdx.x == 0) putStats(a, s);
  if (a.start[a.nranks] == 0) return;   // a launch for the stats alone
  const PolPlace at = polPlace(a);
  if (a.dlogp[at.rank] == nullptr) return;
  const double factor = a.gradScale * partOf(a, s[3]);
  for (int64_t i = at.first; i < at.count; i += at.step) putGrad(a, at.rank, (int)i, factor);
}

// Few tokens: one workgroup, one launch.
__global__ void __launch_bounds__(kPolFewBlock) policyFew(const PolArgs a) {
  __shared__ double lds[kPolFewBlock / kWave][kPolSums];
  double s[kPolSums] = {0.0, 0.0, 0.0, 0.0};
  for (int r = 0; r < a.nranks; ++r)
    for (int i = threadIdx.x; i < a.start[r + 1] - a.start[r]; i += kPolFewBlock) addToken(a, r, i, s);
  blockSums<kPolFewBlock>(s, lds);
  if (threadIdx.x == 0) putStats(a, s);
  const double factor = a.gradScale * partOf(a, s[3]);
  for (int r = 0; r < a.nranks; ++r) {
    if (a.dlogp[r] == nullptr) continue;
    for (int i = threadIdx.x; i < a.start[r + 1] - a.start[r]; i += kPolFewBlock) putGrad(a, r, i, factor);
  }
}

// Workgroups, and partial sums, of a launch of `tokens` tokens.
int polBlocks(int64_t tokens) {
  const int64_t full = (tokens + kPolBlock - 1) / kPolBlock;
  return (int)(full < kPolGrid ? full : kPolGrid);
}

bool polFew(const Shape& s) { return s.total == 0 || (s.launches == 1 && s.total <= kPolFew); }

arResult_t polWorkspace(const size_t* tokens, int nranks, size_t* bytes) {
  Shape s;
  if (bytes == nullptr || !rowsOk(tokens, nranks, &s)) return arInvalidArgument;
  size_t partials = 0;
  if (!polFew(s))
    for (int l = 0; l < s.launches; ++l) {
      const int64_t n = rowsOfLaunch(tokens, nranks, l * kOpRanks);
      const int most = n > 0 ? polBlocks(n) : 0;
      partials += (size_t)(most > 0 && most < kOpRanks ? kOpRanks : most);   // one at least for each rank with tokens
    }
  *bytes = partials * kPolSums * sizeof(double);
  return arSuccess;
}

void fillTokens(PolArgs* a, const float* const* logp, const float* const* old, const float* const* ref,
                const float* const* advantage, const float* const* weight, float* const* dlogp, const size_t* tokens,
                int nranks, int first) {
  a->nranks = nranks - first < kOpRanks ? nranks - first : kOpRanks;
  a->start[0] = 0;
  for (int r = 0; r < a->nranks; ++r) {
    const int k = first + r;
    const bool any = tokens[k] > 0;
    a->start[r + 1] = a->start[r] + (int)tokens[k];
    a->logp[r] = any ? logp[k] : nullptr;
    a->old[r] = any ? old[k] : nullptr;
    a->ref[r] = any && ref ? ref[k] : nullptr;
    a->advantage[r] = any ? advantage[k] : nullptr;
    a->weight[r] = any && weight ? weight[k] : nullptr;
    a->dlogp[r] = any && dlogp ? dlogp[k] : nullptr;
  }
  const int64_t n = a->start[a->nranks];
  if (n > 0) shareOut(a->start, a->nranks, kPolBlock, polBlocks(n), a->blockStart);
  else a->blockStart[a->nranks] = 0;
}

arResult_t policyLoss(const float* const* logp, const float* const* old, const float* const* ref,
                      const float* const* advantage, const float* const* weight, float* const* dlogp,
                      const size_t* tokens, int nranks, double clipLow, double clipHigh, double klCoef,
                      double denominator, double gradScale, float* stats, void* workspace, size_t workspaceGiven,
                      hipStream_t st) {
  Shape s;
  if (!rowsOk(tokens, nranks, &s) || !aligned(stats, 4)) return arInvalidArgument;
  if (!(clipLow >= 0.0 && clipLow <= 1.0) || !(clipHigh >= 0.0)) return arInvalidArgument;
  if (!(klCoef >= 0.0) || !std::isfinite(klCoef) || !std::isfinite(gradScale)) return arInvalidArgument;
  if (!(denominator >= 0.0) || !std::isfinite(denominator)) return arInvalidArgument;
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
  const bool few = polFew(s);
  if (!few) {
    size_t need = 0;
    const arResult_t r = polWorkspace(tokens, nranks, &need);
    if (r != arSuccess) return r;
    if (workspace == nullptr || (uintptr_t)workspace % 16 != 0 || workspaceGiven < need) return arInvalidArgument;
    v.push_back(Extent{(uintptr_t)workspace, need, 1, need, true, -1});
  }
  if (outputsOverlap(v)) return arInvalidArgument;
  PolArgs a{};
  a.low = 1.0 - clipLow;
  a.high = 1.0 + clipHigh;
  a.logLow = std::log1p(-clipLow);
  a.logHigh = std::log1p(clipHigh);
  a.klCoef = klCoef;
  a.denominator = denominator;
  a.gradScale = gradScale;
  if (few) {
    fillTokens(&a, logp, old, ref, advantage, weight, dlogp, tokens, nranks, 0);
    a.stats = stats;
    return launchKernel(policyFew, dim3(1), dim3(kPolFewBlock), a, st) == hipSuccess ? arSuccess : arHipError;
  }
  for (int l = 0; l < s.launches; ++l) {
    fillTokens(&a, logp, old, ref, advantage, weight, dlogp, tokens, nranks, l * kOpRanks);
    a.partials += a.blockStart[a.nranks];
  }
  int partials = 0;
  for (int l = 0; l < s.launches; ++l) {
    fillTokens(&a, logp, old, ref, advantage, weight, dlogp, tokens, nranks, l * kOpRanks);
    const int grid = a.blockStart[a.nranks];
    if (grid == 0) continue;
    a.partial = (double*)workspace + partials;
    if (launchKernel(policySums, dim3(grid), dim3(kPolBlock), a, st) != hipSuccess) return arHipError;
    partials += grid;
  }
  a.partial = (double*)workspace;
  for (int l = 0; l < s.launches; ++l) {
    fillTokens(&a, logp, old, ref, advantage, weight, dlogp, tokens, nranks, l * kOpRanks);
    a.stats = l == 0 ? stats : nullptr;
    const int grid = dlogp != nullptr ? a.blockStart[a.nranks] : 0;
    if (grid == 0 && l > 0) continue;
    if (launchKernel(policyGrad, dim3(grid > 0 ? grid : 1), dim3(kPolBlock), a, st) != hipSuccess) return arHipError;
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
