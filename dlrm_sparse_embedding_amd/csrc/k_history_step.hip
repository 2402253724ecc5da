// Attention of one new item of each history over its slots in a paged cache, with
// the bias by relative position (k_history.hip has the formulas).
//
// Layout. A block takes a sequence, a cache head and a part of the slots; its four
// waves take every fourth tile of 32 slots for the cache head's query heads (at
// most 32, the columns of the product) and are joined in LDS. Keys go straight
// into registers, values through the wave's own LDS tile, both a tile ahead, and
// their pages are looked up another tile ahead. Long histories are split into
// parts, which a second launch joins with the weights 2^(z_i - max z). It is bound
// by reading the slots once: 61 users of up to 3000 slots, 32 x 8 heads of 128
// bf16, 90 us, 4.6 TB/s (75 on the same inputs again, a part of which is still in the
// last cache); one user of 60001, 16 x 4 heads of 64 fp16, 20 us, of which the join is
// 5 and the rest bound by dependent reads (length, page, slot).
#include <algorithm>

#include "history_device.h"

namespace emb {

namespace {

constexpr float kShift = 8.f;  // probabilities carry this many powers of two
constexpr float kSlack = 7.f;  // and this many more before the reference moves
constexpr int kMaxParts = 128;

struct StepDev {
  HistoryStepArgs a;
  float scale2;
  int m;
};

// Where the lane's slot (lane % 32 of a tile) is.
struct Slot {
  int page, in_page;
};

template <int D>
constexpr int kPieces = D / 16;  // 16-byte pieces of 32 rows for each lane

template <int DT, int D, bool BIAS>
__global__ __launch_bounds__(256, 2) void k_history_step(StepDev p) {
  constexpr int OS = D + 4;  // row stride of the joined outputs: rows start 4 banks apart
  constexpr int kV = 4 * 32 * D * 2, kO = (2 * 32 * OS + 4 * 64) * 4;
  __shared__ __attribute__((aligned(1024))) char smem[kV > kO ? kV : kO];
  __shared__ int s_first[BIAS ? EMB_MAX_BUCKETS + 1 : 1];
  __shared__ float s_value[BIAS ? EMB_MAX_BUCKETS : 1][BIAS ? 32 : 1];  // [row][query head of the cache head]
  __shared__ __attribute__((aligned(16))) int s_row[BIAS ? 4 : 1][32];
  const HistoryStepArgs& a = p.a;
  const KvView& kv = a.kv;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = blockIdx.x % a.parts, h = blockIdx.x / a.parts % kv.heads, b = blockIdx.x / (a.parts * kv.heads);
  short* v = reinterpret_cast<short*>(smem) + wave * 32 * D;

  int len = a.lens[b];
  const long long cap = (long long)a.width * kv.page;
  if (len < 0 || len > cap) {
    if (kv.error) atomicOr(kv.error, kKvBadPage);
    len = len < 0 ? 0 : (int)cap;
  }
  len = __builtin_amdgcn_readfirstlane(len);
  // whole rounds of the four waves
  const int chunk = (((len + a.parts - 1) / a.parts) + 127) & ~127;
  const int k0 = (int)min((long long)part * chunk, (long long)len), k1 = min(k0 + chunk, len);
  const int* pages = a.table + (long long)b * a.width;

  auto look = [&](int k) {  // slots past the end repeat the last one; their scores are masked
    const int slot = min(k + (lane & 31), k1 - 1);
    const int col = div_by(kv.by_page, slot);
    return Slot{pages[col], slot - col * kv.page};
  };
  s8v kf[D / 16], vr[kPieces<D>];
  auto load = [&](Slot s) {
    if ((unsigned)s.page >= (unsigned)kv.pages) {
      if (kv.error) atomicOr(kv.error, kKvBadPage);
      s.page = 0;  // in range; what it holds is meaningless
    }
    const short* kp = reinterpret_cast<const short*>(kv.k) + s.page * kv.kps + s.in_page * kv.kss + h * kv.khs;
    // four loads take a line together: they leave it to the caches, unlike those of
    // values (61 users, 8 heads of 128: 119 us with nontemporal ones, now 90)
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      kf[i] = *reinterpret_cast<const s8v*>(kp + 16 * i + 8 * (lane >> 5));
#pragma unroll
    for (int i = 0; i < kPieces<D>; ++i) {
      const int piece = i * 64 + lane, row = piece / (D / 8);
      const int pg = __shfl(s.page, row, 64), at = __shfl(s.in_page, row, 64);
      vr[i] = __builtin_nontemporal_load(reinterpret_cast<const s8v*>(
          reinterpret_cast<const short*>(kv.v) + pg * kv.vps + at * kv.vss + h * kv.vhs + 8 * (piece % (D / 8))));
    }
  };

  const int begin = k0 + 32 * wave;
  Slot next{};
  if (begin < k1) {
    load(look(begin));
    if (begin + 128 < k1) next = look(begin + 128);
  }
  if (BIAS) {
    for (int i = threadIdx.x; i <= a.h.buckets.n; i += 256) s_first[i] = a.h.buckets.first[i];
    for (int i = threadIdx.x; i < a.h.buckets.n * 32; i += 256) {
      const int c = i & 31;
      s_value[i >> 5][c] = c < p.m ? bias_log2(a.bias[(long long)(i >> 5) * a.h.q_heads + h * p.m + c]) : 0.f;
    }
    __syncthreads();
  }
  const int c = min(lane & 31, p.m - 1);  // columns past the last head repeat it; they are not stored
  s8v q[D / 16];
  load_operands<D>(a.q, b, h * p.m + c, q);
  f16v o[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d) o[d] = f16v{};
  float mx = kNegInf, sum = 0.f;
  const TileLane<D> tl;
  const int far_from = BIAS ? a.h.buckets.first[a.h.buckets.n - 1] : 0;

  for (int k = begin; k < k1; k += 128) {
    f16v s[1];
    s[0] = f16v{};
#pragma unroll
    for (int i = 0; i < D / 16; ++i) s[0] = mfma<DT>(kf[i], q[i], s[0]);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the last tile's reads are over
#pragma unroll
    for (int i = 0; i < kPieces<D>; ++i) {
      // values behind the end are cleared: a probability of zero must not meet an infinity
      const int piece = i * 64 + lane, row = piece / (D / 8);
      *reinterpret_cast<s8v*>(v + row * D + 8 * (piece % (D / 8) ^ swizzle<D>(row))) = k + row < k1 ? vr[i] : s8v{};
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (k + 128 < k1) {
      load(next);
      if (k + 256 < k1) next = look(k + 256);
    }
    float mul = p.scale2, add = 0.f;  // a score is s * mul + add
    if (BIAS) {
      if (len - 1 - (k + 31) >= far_from) {
        add = s_value[a.h.buckets.n - 1][lane & 31];
      } else {
        if (lane < 32) s_row[wave][lane] = bucket_of(a.h.buckets, s_first, max(len - 1 - (k + lane), 0));
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[0][i] = fmaf(s[0][i], p.scale2, s_value[s_row[wave][8 * (i / 4) + 4 * (lane >> 5) + i % 4]][lane & 31]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        mul = 1.f;
      }
    }
    if (k + 32 > k1) mask_tile(s[0], k, k1);
    const float top = fmaf(both_halves_max(top_of(s)), mul, add);
    const bool up = top > mx + kSlack;
    if (__ballot(up)) {
      const float keep = up ? __builtin_amdgcn_exp2f(mx - top) : 1.f;
      mx = up ? top : mx;
      sum *= keep;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= keep;
    }
    add += kShift - (mx == kNegInf ? 0.f : mx);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[0][i] = __builtin_amdgcn_exp2f(fmaf(s[0][i], mul, add));
      sum += s[0][i];
    }
    s8v w[2];
    pack_tile<DT>(s[0], w);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int d = 0; d < D / 32; ++d) o[d] = mfma<DT>(tl.columns(v, 16 * kk, d), w[kk], o[d]);
  }

  // join: waves 2 and 3 into 0 and 1, then 1 into 0
  float* so = reinterpret_cast<float*>(smem);
  float* sm = so + 2 * 32 * OS;
  for (int half = 2; half >= 1; half >>= 1) {
    __syncthreads();
    if (wave >= half && wave < 2 * half) {
      float* dst = so + (wave - half) * 32 * OS + (lane & 31) * OS + 4 * (lane >> 5);
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<f4*>(dst + 32 * d + 8 * i) = f4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
      sm[(wave - half) * 128 + lane] = mx;
      sm[(wave - half) * 128 + 64 + lane] = sum;
    }
    __syncthreads();
    if (wave < half) {
      const float omx = sm[wave * 128 + lane], osum = sm[wave * 128 + 64 + lane];
      const float top = fmaxf(mx, omx);
      const float ka = top == kNegInf ? 1.f : __builtin_amdgcn_exp2f(mx - top);
      const float kb = top == kNegInf ? 0.f : __builtin_amdgcn_exp2f(omx - top);
      mx = top;
      sum = sum * ka + osum * kb;
      const float* src = so + wave * 32 * OS + (lane & 31) * OS + 4 * (lane >> 5);
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f4 x = *reinterpret_cast<const f4*>(src + 32 * d + 8 * i);
#pragma unroll
          for (int j = 0; j < 4; ++j) o[d][4 * i + j] = o[d][4 * i + j] * ka + x[j] * kb;
        }
    }
  }
  if (wave > 0) return;
  const float total = both_halves_sum(sum);
  const bool some = !(total == 0.f);  // a NaN counts
  const float z = some ? mx - kShift + __log2f(total) : kNegInf;
  const float inv = some ? 1.f / total : 0.f;
  const bool store = (lane & 31) < p.m;
  const int head = h * p.m + c;
  if (a.parts == 1) {
    if (a.lse && store && lane < 32) a.lse[(long long)b * a.h.q_heads + head] = some ? z * kLn2 : kNegInf;
    if (!some) {
#pragma unroll
      for (int d = 0; d < D / 32; ++d) o[d] = f16v{};
    }
    short* dst = reinterpret_cast<short*>(const_cast<void*>(a.out.p)) + b * a.out.ts + head * a.out.hs + 8 * (lane >> 5);
    store_columns<DT, D>(dst, o, inv, store);
    return;
  }
  if (!store) return;
  const long long at = ((long long)part * a.seqs + b) * a.h.q_heads + head;
  if (lane < 32) a.part_lse[at] = z;
  if (!some) return;
  float* dst = a.part_o + at * D + 4 * (lane >> 5);
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<f4*>(dst + 32 * d + 8 * i) =
          f4{o[d][4 * i] * inv, o[d][4 * i + 1] * inv, o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv};
}

// Joins the parts of each (sequence, query head). A row is taken by GROUPS (1 or 8)
// groups of 32 lanes, 4 columns a lane, each of which takes every GROUPS-th set of
// eight parts (128 parts of 16 rows of 64: 17.7 us with one, 5.2 with eight).
template <int DT, int D, int GROUPS>
__global__ __launch_bounds__(256) void k_history_join(StepDev p) {
  const HistoryStepArgs& a = p.a;
  const int l = threadIdx.x & 31, group = threadIdx.x >> 5;
  const long long rows = (long long)a.seqs * a.h.q_heads;
  const long long row = GROUPS == 1 ? (long long)blockIdx.x * 8 + group : blockIdx.x;
  if (row >= rows) return;
  float z[kMaxParts / 32], top = kNegInf;
#pragma unroll
  for (int i = 0; i < kMaxParts / 32; ++i) {
    z[i] = l + 32 * i < a.parts ? a.part_lse[(l + 32 * i) * rows + row] : kNegInf;
    top = fmaxf(top, z[i]);
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 32));
  const float ref = top == kNegInf ? 0.f : top;
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxParts / 32; ++i) {
    z[i] = __builtin_amdgcn_exp2f(z[i] - ref);
    total += z[i];
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) total += __shfl_xor(total, d, 32);
  f4 acc = {0.f, 0.f, 0.f, 0.f};
  // eight parts' loads at once; an empty part holds nothing, not zeros
#pragma unroll
  for (int g = 0; g < kMaxParts / 32; ++g)
    for (int i = 32 * g + (GROUPS == 1 ? 0 : 8 * (group & 3)); i < min(a.parts, 32 * g + 32); i += GROUPS == 1 ? 8 : 32) {
      if (GROUPS > 1 && (g & 1) != (group >> 2)) continue;
      f4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        x[k] = *reinterpret_cast<const f4*>(a.part_o + (min(i + k, a.parts - 1) * rows + row) * D + 4 * min(l, D / 4 - 1));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float w = __shfl(z[g], i - 32 * g + k, 32);
        if (i + k < a.parts && w != 0.f) acc += x[k] * w;
      }
    }
  if constexpr (GROUPS > 1) {
    __shared__ f4 s_acc[GROUPS][32];
    s_acc[group][l] = acc;
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) acc += s_acc[g][l];
  }
  const bool some = !(total == 0.f);
  const float inv = some ? 1.f / total : 0.f;
  const long long b = row / a.h.q_heads;
  const int head = (int)(row - b * a.h.q_heads);
  if (l < D / 4) {
    const u2 x = {pack2<DT>(acc.x * inv, acc.y * inv), pack2<DT>(acc.z * inv, acc.w * inv)};
    *reinterpret_cast<u2*>(reinterpret_cast<short*>(const_cast<void*>(a.out.p)) + b * a.out.ts + head * a.out.hs + 4 * l) = x;
  }
  if (l == 0 && a.lse) a.lse[row] = some ? (top + __log2f(total)) * kLn2 : kNegInf;
}

template <int DT, int D>
hipError_t launch(const StepDev& p, hipStream_t st) {
  const HistoryStepArgs& a = p.a;
  const unsigned blocks = (unsigned)((long long)a.seqs * a.kv.heads * a.parts);
  if (a.bias) k_history_step<DT, D, true><<<blocks, 256, 0, st>>>(p);
  else k_history_step<DT, D, false><<<blocks, 256, 0, st>>>(p);
  if (hipError_t e = hipGetLastError()) return e;
  if (a.parts == 1) return hipSuccess;
  // many parts are those of few sequences
  const long long rows = (long long)a.seqs * a.h.q_heads;
  if (a.parts > 16) k_history_join<DT, D, 8><<<(unsigned)rows, 256, 0, st>>>(p);
  else k_history_join<DT, D, 1><<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace

// Parts of the slots, by the table's width, since lengths are on the device: as many
// as make 1024 blocks, but no more than the width has runs of 256 slots, since each
// part writes and reads back an fp32 partial output. A sequence shorter than the
// width has parts of whole rounds of the four waves, 128 slots, and empty ones. (61
// users of up to 3000 slots, 488 pairs with a head: 89 us, 95 for 600 blocks, 96 for
// 1500, 97 for 2048; 200 users of up to 1000: 88, 88, 88 and 114; 4 of up to 20000:
// 45, 43, 50 and 56.)
int history_step_parts(const HistoryView& h, const KvView& kv, int seqs, int width) {
  const long long items = (long long)seqs * h.kv_heads, cap = (long long)width * kv.page;
  if (items == 0) return 1;
  const long long want = (1024 + items - 1) / items;
  return (int)std::max<long long>(1, std::min<long long>({want, (cap + 255) / 256, (long long)kMaxParts}));
}

hipError_t launch_history_step(const HistoryStepArgs& a, hipStream_t st) {
  StepDev p{};
  p.a = a;
  p.scale2 = a.h.scale * kLog2e;
  p.m = a.h.q_heads / a.h.kv_heads;
  const bool bf = a.h.dtype == EMB_BF16;
  switch (a.h.dim) {
    case 64: return bf ? launch<EMB_BF16, 64>(p, st) : launch<EMB_F16, 64>(p, st);
    case 96: return bf ? launch<EMB_BF16, 96>(p, st) : launch<EMB_F16, 96>(p, st);
    default: return bf ? launch<EMB_BF16, 128>(p, st) : launch<EMB_F16, 128>(p, st);
  }
}

}  // namespace emb
