// Launch parameters, work plan and launchers of the latent-attention kernels (internal).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"

namespace v4a {

constexpr int kRotMaxPairs = 128;

// A rotation's turning rates as turns per position, phi_i and psi_i = frac(4096 phi_i), each
// split into fp32 hi + lo on the host (in double), as in Rope.
struct RotTab {
  int32_t dim, layout;
  float amp;
  float phi_hi[kRotMaxPairs], phi_lo[kRotMaxPairs];
  float psi_hi[kRotMaxPairs], psi_lo[kRotMaxPairs];
};

struct RopeParams {
  int32_t n_tokens, n_heads, inverse;
  const int64_t* pos;
  const void* x;
  void* y;
  int64_t x_ts, x_hs, y_ts, y_hs;
  int32_t* err;
  RotTab rot;
};

struct LatentInsertParams {
  int32_t n_seq, n_tokens, C;
  const int32_t* cu;
  const int64_t* start;
  const void* c;
  const void* k_pe;
  int64_t c_stride, k_stride;
  const float* gamma;
  float eps;
  CacheView cache;
  int32_t* err;
  RotTab rot;
};

struct LatentGatherParams {
  int32_t n_seq, n_rows, row_bytes;
  const int32_t* cu;
  const int64_t* start;
  CacheView cache;
  void* out;
  int32_t* err;
};

// The work of an absorbed call. The rows (token, head) of a sequence are consecutive rows of
// q; they are cut into units of NR rows, and the sequence's keys into tiles of TK. Lengths are
// known on the device only, so every CTA derives the plan from cu and start: U consecutive
// units of a sequence form a share (its members walk the same key tiles at the same time and
// meet in L2), CTAs in teams of U take equal parts of all (share, tile) pairs in order. A unit
// whose tiles fall to several teams is left as partial results that a second kernel merges.
// U is 1, 2 or 4, at most max_U, the largest that costs no more than 1/8 in members without a
// unit. Without a split, whole units go to the CTAs in turn and nothing is merged: the host knows
// that it has many units, but not whether one of them is as long as many others together, so
// there the device decides.
constexpr int32_t kSplitNone = 0, kSplitAll = 1, kSplitOnDevice = 2;
struct LatentPlan {
  int32_t NR, TK;
  int32_t max_U;
  int32_t ctas;                       // of the launch, a multiple of max_U
  int32_t split;                      // kSplit*; the workspace and the merge go with all but None
  int32_t split_ctas;                 // the CTAs that work where units are split (<= ctas, a multiple
                                      // of max_U): each may leave two partial results
  int32_t tc;                         // tensor-core kernel
};

struct LatentAttnParams {
  int32_t n_seq, n_tokens, H, C, R;   // R = rotary dims
  float scale;
  int64_t max_pos;
  int64_t end;                        // no key is at or behind it: max_pos + 1 and the table's reach
  const int32_t* cu;
  const int64_t* start;
  const void* q;
  void* out;
  CacheView cache;
  LatentPlan plan;
  float* part_o;                      // [split_ctas][2][NR][C] unnormalised, fp32
  float* part_ml;                     // [split_ctas][2][NR][2] reference (log2 units) and sum
  int32_t* part_job;                  // [split_ctas][4] what to merge (LatentWalk::post)
  int32_t* err;
};

struct LatentExpandedParams {
  int32_t n_seq, n_q, n_k, H, DN, DR, DV, causal;
  float scale;
  const int32_t* cu_q;
  const int32_t* cu_k;
  const void* q;
  const void* k;
  const void* k_pe;
  const void* v;
  void* out;
  int64_t k_ts, k_hs, pe_ts, v_ts, v_hs;
  // tensor-core kernel: pairs of CTAs, whether items may be split among them, steps that starting
  // an item counts for (0 without split: then every item is one step and no pair gets part of
  // one, so the partial results' pointers are not used), partial results
  int32_t tc, pairs, split, setup;
  float* part_o;                      // [pairs][2][512][128] unnormalised, fp32
  float* part_ml;                     // [pairs][2][512][2] reference (log2 units) and sum
  int32_t* part_job;                  // [pairs][8] what to merge
  int32_t* err;
};

// SMs of the current device (152, a GB300's, where there is none to ask).
int sm_count();
int launch_rope(const RopeParams& p, int dtype, cudaStream_t st);
int launch_latent_insert(const LatentInsertParams& p, int dtype, cudaStream_t st);
int launch_latent_gather(const LatentGatherParams& p, cudaStream_t st);
int launch_latent_attn(const LatentAttnParams& p, int dtype, cudaStream_t st);
int launch_latent_expanded(const LatentExpandedParams& p, int dtype, cudaStream_t st);
cudaError_t launch_latent_attn_tc(const LatentAttnParams& p, cudaStream_t st);
cudaError_t launch_latent_expanded_tc(const LatentExpandedParams& p, cudaStream_t st);
cudaError_t launch_latent_merge(const LatentAttnParams& p, int dtype, cudaStream_t st);

// ------------------------------------------------------------------ device-side plan
#ifdef __CUDACC__

// Rows of a packed batch that belong to sequence b, inside [0, n) whatever cu holds.
__device__ __forceinline__ int cu_at(const int32_t* cu, int i, int n) {
  return min(max(__ldg(cu + i), 0), n);
}

// Sequence of packed row t: the last b with cu[b] <= t, or -1 when t is outside the batch.
__device__ __forceinline__ int find_seq(const int32_t* cu, int n_seq, int t) {
  int lo = 0, hi = n_seq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid; else hi = mid;
  }
  return t >= __ldg(cu + lo) && t < __ldg(cu + lo + 1) ? lo : -1;
}

// One sequence's part of the plan.
struct LatentSeq {
  int row0;          // first row of the batch's (token, head) rows
  int rows;          // rows of the sequence
  int units;         // units of NR rows
  int tiles;         // key tiles of the whole sequence (1 in whole-unit plans)
  int64_t start;     // position of its first new token
  __device__ __forceinline__ int shares(int U) const { return (units + U - 1) / U; }
  __device__ __forceinline__ int pairs(int U) const { return shares(U) * tiles; }
};

__device__ __forceinline__ LatentSeq latent_seq(const LatentAttnParams& p, int b, bool split) {
  LatentSeq s;
  const int a = cu_at(p.cu, b, p.n_tokens);
  const int n = max(cu_at(p.cu, b + 1, p.n_tokens) - a, 0);
  s.row0 = a * p.H;
  s.rows = n * p.H;
  s.start = __ldg(p.start + b);
  s.units = (s.rows + p.plan.NR - 1) / p.plan.NR;
  const int64_t keys = min(s.start + n, p.end);
  s.tiles = !split || keys <= 0 ? 1 : (int)((keys + p.plan.TK - 1) / p.plan.TK);
  return s;
}

// Keys that a token at pos sees (0 for a position below 0).
__device__ __forceinline__ int64_t latent_visible(const LatentAttnParams& p, int64_t pos) {
  return max((int64_t)0, min(pos, p.end - 1) + 1);
}
// What is to be reported of a token's position. (Positions that the block table does not reach are
// blocks without a page; only the table's are walked.)
__device__ __forceinline__ void latent_report_pos(const LatentAttnParams& p, int64_t pos) {
  if (pos > p.max_pos || pos < 0) raise_err(p.err, V4A_DEV_BAD_POS);
  if (min(pos, p.max_pos) >= p.end) raise_err(p.err, V4A_DEV_MISSING_PAGE);
}
// The same for token i of a sequence.
__device__ __forceinline__ int64_t latent_visible(const LatentAttnParams& p, const LatentSeq& s, int i) {
  return latent_visible(p, s.start + i);
}

// Exclusive prefix sums of weight(b) over the sequences into pre[0 .. n_seq] (shared memory),
// by the whole block.
template <typename F>
__device__ __forceinline__ void seq_prefix(int n_seq, int32_t* pre, int32_t* warp_tot, F weight) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int carry = 0;
  for (int b0 = 0; b0 < n_seq; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    const int w = b < n_seq ? weight(b) : 0;
    int x = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_tot[warp] = x;
    __syncthreads();
    int before = carry, all = 0;
    for (int i = 0; i < nw; ++i) {
      if (i < warp) before += warp_tot[i];
      all += warp_tot[i];
    }
    if (b < n_seq) pre[b] = before + x - w;
    carry += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) pre[n_seq] = carry;
  __syncthreads();
}
// Whether the call's units are split along the keys, by the whole block (alike in every block).
// Of many units, whole ones take an even part of the tiles that they see and about half the longest
// unit more; split ones take an even part of a line in which every unit counts as long as its
// sequence's last one (in prompts up to twice what they see). The shorter is taken. 64 heads, whole
// and split: a 2,048-token prompt 429 and 680 us, 700 tokens 90 and 119; 1,000 tokens after 3,000
// beside eight decode tokens on 20,000 each 944 and 701; 606 beside one on 100,000: 2151 and 137.
__device__ __forceinline__ bool latent_split(const LatentAttnParams& p, int32_t* warp_tot) {
  if (p.plan.split != kSplitOnDevice) return p.plan.split == kSplitAll;
  int sees = 0, line = 0, longest = 0;
  for (int b = threadIdx.x; b < p.n_seq; b += blockDim.x) {
    const LatentSeq s = latent_seq(p, b, true);
    if (s.units == 0) continue;
    const int first = (int)((latent_visible(p, s, 0) + p.plan.TK - 1) / p.plan.TK);
    sees += s.units * ((first + s.tiles + 1) / 2);
    line += s.units * s.tiles;
    longest = max(longest, s.tiles);
  }
  if (threadIdx.x < 3) warp_tot[threadIdx.x] = 0;
  __syncthreads();
  sees = __reduce_add_sync(0xffffffffu, sees);
  line = __reduce_add_sync(0xffffffffu, line);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if ((threadIdx.x & 31) == 0 && longest > 0) {
    atomicAdd(warp_tot, sees);
    atomicAdd(warp_tot + 1, line);
    atomicMax(warp_tot + 2, longest);
  }
  __syncthreads();
  const int64_t whole2 = 2 * (int64_t)warp_tot[0] + (int64_t)warp_tot[2] * p.plan.split_ctas;
  const bool split = whole2 > 2 * (int64_t)warp_tot[1];
  __syncthreads();
  return split;
}

// U and the (share, tile) pairs before each sequence of an absorbed call, by the whole block.
__device__ __forceinline__ int latent_prefix(const LatentAttnParams& p, bool split, int32_t* pre,
                                             int32_t* warp_tot) {
  int U = p.plan.max_U;
  if (U > 1) {
    int c1 = 0, c2 = 0, c4 = 0;
    for (int b = threadIdx.x; b < p.n_seq; b += blockDim.x) {
      const LatentSeq s = latent_seq(p, b, split);
      c1 += s.pairs(1);
      c2 += s.pairs(2);
      c4 += s.pairs(4);
    }
    if (threadIdx.x < 3) warp_tot[threadIdx.x] = 0;
    __syncthreads();
    c1 = __reduce_add_sync(0xffffffffu, c1);
    c2 = __reduce_add_sync(0xffffffffu, c2);
    c4 = __reduce_add_sync(0xffffffffu, c4);
    if ((threadIdx.x & 31) == 0 && c1 > 0) {
      atomicAdd(warp_tot, c1);
      atomicAdd(warp_tot + 1, c2);
      atomicAdd(warp_tot + 2, c4);
    }
    __syncthreads();
    c1 = warp_tot[0];
    c2 = warp_tot[1];
    c4 = warp_tot[2];
    __syncthreads();
    const int most = c1 + c1 / 8;
    if (U == 4 && (int64_t)c4 * 4 > most) U = 2;
    if (U == 2 && (int64_t)c2 * 2 > most) U = 1;
  }
  seq_prefix(p.n_seq, pre, warp_tot, [&](int b) { return latent_seq(p, b, split).pairs(U); });
  return U;
}

// The sequence that holds position x of the prefix sums (pre[b] <= x < pre[b + 1]).
__device__ __forceinline__ int latent_seq_at(const int32_t* pre, int n_seq, int x) {
  int lo = 0, hi = n_seq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Team g takes pairs [g * per, (g + 1) * per) of a line of `total`, with the smallest per that n
// teams can do with: no team more than in an even split, fewer teams where they suffice, and cuts
// that fall together with those of equally long units where per divides their length.
__device__ __forceinline__ int latent_per_team(int total, int n) { return n > 0 ? (total + n - 1) / n : 1; }

// One piece of work of a CTA: a unit and a range of its key tiles.
struct LatentPiece {
  int seq, row0, rows;         // row0: first row of the unit in q; rows <= NR
  int tile0, tile1;            // key tiles of the sequence
  int64_t keys, keys0;         // keys that the unit's last and first rows see
  int64_t start;               // position of the sequence's first token
  int seq_row0;                // first row of the sequence
  int whole;                   // the piece holds every tile of the unit: write the result
  int slot;                    // where its partial result goes otherwise
  int job_rows, job_last;      // set where the piece is the second of its unit's pieces (see below)
};

// Walks a CTA's pieces, forward through the sequences. All threads of a role call it alike;
// the prefix sums are read in begin() only.
struct LatentWalk {
  int x, x1, cta, team, member, U, n, per;   // n: stride of whole shares (0: split ones); per: pairs of a team
  int b, base;      // current sequence and the pairs before it
  // The plan, in pre (shared memory) and here, by the whole block.
  __device__ __forceinline__ void begin(const LatentAttnParams& p, int32_t* pre, int32_t* warp_tot) {
    const bool split = latent_split(p, warp_tot);
    U = latent_prefix(p, split, pre, warp_tot);
    cta = blockIdx.x;
    const int total = pre[p.n_seq];
    team = cta / U;
    member = cta % U;
    const int teams = (split ? p.plan.split_ctas : p.plan.ctas) / U;
    per = latent_per_team(total, teams);
    if (!split) {                  // whole shares in turn, the teams striding over them
      n = teams;
      x = team;
      x1 = total;
    } else {
      n = 0;
      x = team < teams ? min(team * per, total) : 0;
      x1 = team < teams ? min(x + per, total) : 0;
    }
    b = x < x1 ? latent_seq_at(pre, p.n_seq, x) : 0;
    base = x < x1 ? pre[b] : 0;
  }
  // A team's merge job, if any, is its first piece's: every team posts one, empty or not,
  // before that piece's results (an empty one too where the device decided against a split).
  __device__ __forceinline__ void post(const LatentAttnParams& p, const LatentPiece* w) const {
    if (p.plan.split == kSplitNone || cta >= p.plan.split_ctas) return;
    const int rows = w ? w->job_rows : 0;
    *reinterpret_cast<int4*>(p.part_job + 4 * cta) =
        make_int4(rows, rows > 0 ? w->row0 : 0, rows > 0 ? w->job_last : 0, U);
  }
  // The next piece, or false. A piece may have no unit (rows == 0) or no keys.
  __device__ __forceinline__ bool next(const LatentAttnParams& p, LatentPiece& w) {
    if (x >= x1) return false;
    LatentSeq s = latent_seq(p, b, n == 0);
    while (b + 1 < p.n_seq && x >= base + s.pairs(U)) {
      base += s.pairs(U);
      s = latent_seq(p, ++b, n == 0);
    }
    const int r = x - base;
    const int share = r / s.tiles, t = r - share * s.tiles;
    w.seq = b;
    w.start = s.start;
    w.seq_row0 = s.row0;
    const int unit = share * U + member, ur = unit * p.plan.NR;
    w.row0 = s.row0 + ur;
    w.rows = max(0, min(p.plan.NR, s.rows - ur));
    w.keys = w.rows > 0 ? latent_visible(p, s, (ur + w.rows - 1) / p.H) : 0;
    w.keys0 = w.rows > 0 ? latent_visible(p, s, ur / p.H) : 0;
    const int unit_tiles = (int)((w.keys + p.plan.TK - 1) / p.plan.TK);
    if (n > 0) {
      w.tile0 = 0;
      w.tile1 = unit_tiles;
      w.whole = 1;
      w.slot = 0;
      w.job_rows = 0;
      x += n;
    } else {
      const int take = min(s.tiles - t, x1 - x);
      w.whole = take == s.tiles;
      w.slot = (cta << 1) + (t == 0 ? 1 : 0);
      w.tile0 = min(t, unit_tiles);
      w.tile1 = min(t + take, unit_tiles);
      // The team that holds the second piece of a unit posts the unit's merge: teams team - 1
      // to job_last hold its pieces, in slot 1 of the first and slot 0 of the others.
      const int x0 = x - t;
      const bool second = t > 0 && (team - 1) * per <= x0;
      w.job_rows = second ? w.rows : 0;
      w.job_last = second ? (x0 + s.tiles - 1) / per : 0;
      x += take;
    }
    return true;
  }
};

// Angle of position pos (0 <= pos < 2^36) and a pair's constants: pos = 4096 hi + lo, the
// angle in turns is frac(hi psi + lo phi). Products are exact in two floats, the integer parts
// are dropped exactly, and what the reduced angle loses to rounding turns the result by its
// first-order term, so cosine and sine of these rates are good to a few units of 2^-24. The rates
// themselves are 64-bit numbers of a few roundings: against the exact ones an angle is off by up
// to 12 2^-53 of its position besides (rates 1 .. 1e-4: 1.6 units up to 2^30, 4 at 2^32, 54 at 2^36).
__device__ __forceinline__ void rot_cs(int64_t pos, float phi_hi, float phi_lo, float psi_hi, float psi_lo,
                                       float& c, float& s) {
  const float hi = (float)(int32_t)(pos >> 12), lo = (float)(int32_t)(pos & 4095);
  const float p1 = hi * psi_hi, e1 = fmaf(hi, psi_lo, fmaf(hi, psi_hi, -p1));
  const float p2 = lo * phi_hi, e2 = fmaf(lo, phi_lo, fmaf(lo, phi_hi, -p2));
  const float r1 = p1 - rintf(p1), r2 = p2 - rintf(p2);
  float a = r1 + r2;
  const float bb = a - r1;
  const float tail = ((r1 - (a - bb)) + (r2 - bb)) + (e1 + e2);
  a -= rintf(a);
  const float t = a + tail, d = (tail - (t - a)) * 6.2831853071795865f;
  float c0, s0;
  sincospif(2.0f * t, &s0, &c0);
  c = fmaf(-s0, d, c0);
  s = fmaf(c0, d, s0);
}

#endif  // __CUDACC__

}  // namespace v4a
