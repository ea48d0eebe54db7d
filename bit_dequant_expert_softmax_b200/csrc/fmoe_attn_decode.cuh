// Single-token attention over the paged 4-bit cache (sm_100a).
//
// Per sequence and key/value head, for its G query heads q and len cached tokens j:
//   s_j = scale q . k_j,   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),   m = max_j s_j
// with k_jc = a_jg c_jc + b_jg (code c, one scale a and bias b per 64-channel group g) and v
// likewise, in one pass over the cache with the running maximum and sum per query.
//
// The cache is read once, so the bytes (144 per token and head at D = 128) bound the call; the
// work beside them is turning codes into matrix operands.  Both products run on mma.sync
// m16n8k16 with the cache as the 16-row operand and 8 queries as the columns: one query
// token has at most G rows of work per key, and the tcgen05 forms (64 or 128 rows from shared
// or tensor memory) would need every dequantised operand written to memory again.
//   codes    enter as the exact bf16 1 + c/16 (one rotate and one LOP3 per pair)
//   scores   per group D = sum_c (1 + c/16) q_c, X = sum_c q_c:  sum_c k_c q_c = 16 a D + (b - 16 a) X
//   values   the weights enter as p' = bf16(p a), per group.  With c - 8 as the code's centre
//            p (a c + b) = p' (c - 8) + p (b + 8 a), and sum p' (c - 8) = 16 sum p' (1 + c/16) -
//            24 sum p': only the centred part carries p' 's rounding, so it weighs no more than
//            rounding p does with bf16 values.  Sums, maxima and the b part are fp32.
// A warp's scores leave the first product with keys in rows; movmatrix turns 8x8 blocks of
// the packed weights into the second product's column operand.
//
// Split: the (sequence, key/value head, query block, 64-key step) units of the batch form one
// line that is cut into equal ranges, one per block, found from the lengths on the device (so a
// captured graph follows growing lengths).  A block's part of one sequence and head is a
// segment; its tiles of 16 keys go to the warps in equal runs.  Each warp streams its tiles
// through its own ring of bulk copies, with its own running maximum; warps join in shared
// memory at the segment's end.  A segment that is a whole (sequence, head) is written to the
// output, other segments to the workspace, where a second kernel joins them.
#pragma once

#include "fmoe_kv.cuh"

namespace fmoe {

constexpr int kAdWarps = 4;
constexpr int kAdThreads = kAdWarps * 32;
constexpr int kAdStepTiles = 4;                        // tiles a warp takes at once
constexpr int kAdStep = kAdStepTiles * kKvTile;        // keys of a unit
constexpr int kAdStages = 2;                           // ring slots per warp
constexpr int kAdMaxBlocks = 512;
constexpr unsigned long long kAdWaitNs = 2000000000ull;

// What a block leaves for the joining kernel: it ended a segment that began in block
// `first` (-1: none).
struct AdRecord {
  int first, seq, head0, queries;
};

struct AdParams {
  const uint16_t* q;
  long long q_stride;
  const uint8_t* cache;
  long long pages, page_bytes;
  const int32_t *table, *lens;
  uint16_t* out;
  AdRecord* rec;    // [blocks]
  float* part;      // [blocks][2][queries][D]
  float* part_ml;   // [blocks][2][queries][2]
  uint32_t* err;
  float scale_log2; // scale * log2(e)
  int width, seqs, q_heads, kv_heads, group, qblocks, page_tokens;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// codes i and i + 4 of a word as bf16 1 + c/16
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i) {
  return (__funnelshift_r(w, w, (4 * i - 3) & 31) & 0x00780078u) | 0x3F803F80u;
}

__device__ __forceinline__ int ad_len(const AdParams& p, int s) {
  const int len = __ldg(p.lens + s);
  const long long most = static_cast<long long>(p.width) * p.page_tokens;
  return len <= 0 ? 0 : len > most ? static_cast<int>(most) : len;
}

template <int D, int NT>
struct AdGeom {
  static constexpr int kTile = KvGeom<D>::kTileBytes;
  static constexpr int kStage = kAdStepTiles * kTile;
  static constexpr int kRegs = 16 * KvGeom<D>::kGroups * NT;  // output floats of a thread
  static constexpr int kMerge = 32 * (kRegs + 4 * NT) * 4;    // a warp's state, bytes
  static constexpr int kRing = kAdWarps * kAdStages * kStage;
  static constexpr int kSmem = kRing + kAdWarps / 2 * kMerge + kAdWarps * kAdStages * 8;
};

// One place in the block's line of units, the same in all of its warps.
struct AdCursor {
  long long left;    // units of the block not yet in a segment
  int seq, hb;       // the next segment's sequence and (head, query block)
  int step;          // its first 64-key step
  int len, steps;    // of `seq`
};

template <int D, int NT>
struct AdWarp {
  using Kv = KvGeom<D>;
  using Gm = AdGeom<D, NT>;
  static constexpr int NG = Kv::kGroups;
  const AdParams& p;
  const int warp, lane, g, t;
  const int hbs;               // (head, query block) pairs per sequence
  uint8_t* ring;
  uint64_t* bars;
  float* merge;
  bool lost = false;           // a copy's wait ran out

  // online softmax state: columns 2t and 2t + 1 of every 8-query tile
  float m[NT][2], l[NT][2];
  float off[NT][NG][2];        // sum p (b + 8a) - 24 sum p'
  float o[NT][NG][4][4];
  uint32_t qf[NT][NG][8];      // query fragments
  float X[NT][NG][2];          // group sums of the queries of columns 2t, 2t + 1

  __device__ AdWarp(const AdParams& pp, uint8_t* smem)
      : p(pp), warp(threadIdx.x >> 5), lane(threadIdx.x & 31), g(lane >> 2), t(lane & 3), hbs(pp.kv_heads * pp.qblocks) {
    ring = smem + warp * kAdStages * Gm::kStage;
    merge = reinterpret_cast<float*>(smem + Gm::kRing);
    bars = reinterpret_cast<uint64_t*>(smem + Gm::kRing + kAdWarps / 2 * Gm::kMerge) + warp * kAdStages;
  }

  // tile range of this warp in the segment of steps [a, b)
  __device__ __forceinline__ void run(int len, int a, int b, int& lo, int& hi) const {
    const int t0 = a * kAdStepTiles, t1 = min(b * kAdStepTiles, (len + kKvTile - 1) / kKvTile);
    const int per = (t1 - t0 + kAdWarps - 1) / kAdWarps;
    lo = min(t1, t0 + warp * per);
    hi = min(t1, lo + per);
  }

  // the next segment; false at the end of the block's range
  __device__ __forceinline__ bool next(AdCursor& c, int& seq, int& hb, int& len, int& a, int& b) const {
    if (c.left <= 0) return false;
    seq = c.seq;
    hb = c.hb;
    len = c.len;
    a = c.step;
    b = static_cast<int>(min(static_cast<long long>(c.steps), a + c.left));
    c.left -= b - a;
    c.step = 0;
    if (b == c.steps && c.left > 0 && ++c.hb == hbs) {
      c.hb = 0;
      do {
        if (++c.seq >= p.seqs) {  // not reached while the lengths stay as they are
          c.left = 0;
          return true;
        }
        c.len = ad_len(p, c.seq);
      } while (c.len == 0);
      c.steps = (c.len + kAdStep - 1) / kAdStep;
    }
    return true;
  }

  // Copies of tiles [lo, lo + n) (n <= kAdStepTiles) into ring slot `slot`: a lane per tile.
  // A bad page's tile is not copied; the bits of those that are come back.
  __device__ __forceinline__ uint32_t fetch(int seq, int hb, int lo, int n, uint32_t slot) {
    const uint8_t* src = nullptr;
    if (lane < n) {
      const int tpp = p.page_tokens / kKvTile, tile = lo + lane;
      const int page = __ldg(p.table + static_cast<long long>(seq) * p.width + tile / tpp);
      if (page >= 0 && page < p.pages)
        src = p.cache + page * p.page_bytes +
              (static_cast<long long>(hb / p.qblocks) * tpp + tile % tpp) * static_cast<long long>(Gm::kTile);
      else
        kv_error(p.err, FMOE_DEVERR_BAD_PAGE);
    }
    const uint32_t ok = __ballot_sync(0xffffffffu, src != nullptr);
    if (lane == 0) mbar_arrive_expect_tx(&bars[slot], __popc(ok) * Gm::kTile);
    __syncwarp();
    if (src != nullptr) bulk_g2s(ring + slot * Gm::kStage + lane * Gm::kTile, src, Gm::kTile, &bars[slot]);
    return ok;
  }

  __device__ __forceinline__ void wait(uint32_t slot, uint32_t parity) {
    if (mbar_try_wait(&bars[slot], parity) || lost) return;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(&bars[slot], parity)) {
      if (global_timer_ns() - t0 > kAdWaitNs) {
        lost = true;
        kv_error(p.err, FMOE_DEVERR_COPY_TIMEOUT);
        return;
      }
    }
  }

  // query fragments and group sums of (sequence, head, query block); fresh softmax state
  __device__ __forceinline__ void start(int seq, int hb) {
    const int kvh = hb / p.qblocks, q0 = (hb % p.qblocks) * 8 * NT;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int qi = q0 + nt * 8 + g;
      const bool live = qi < p.group;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + seq * p.q_stride + static_cast<long long>(kvh * p.group + qi) * D);
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        const uint4 a = live ? __ldg(src + n * 8 + 2 * t) : z, b = live ? __ldg(src + n * 8 + 2 * t + 1) : z;
        // channels (i, i + 4) of a word's eight in one register, as the codes' pairs
        const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          qf[nt][n][4 * w] = __byte_perm(x[4 * w], x[4 * w + 2], 0x5410);
          qf[nt][n][4 * w + 1] = __byte_perm(x[4 * w], x[4 * w + 2], 0x7632);
          qf[nt][n][4 * w + 2] = __byte_perm(x[4 * w + 1], x[4 * w + 3], 0x5410);
          qf[nt][n][4 * w + 3] = __byte_perm(x[4 * w + 1], x[4 * w + 3], 0x7632);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += bf16_lo(x[i]) + bf16_hi(x[i]);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        X[nt][n][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
        X[nt][n][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
        off[nt][n][0] = off[nt][n][1] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][n][i][e] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[nt][c] = -INFINITY;
        l[nt][c] = 0.f;
      }
    }
  }

  // tiles in ring slot `slot`: n of them, those of `ok` copied; key0 = the first's token
  __device__ __forceinline__ void step(uint32_t slot, int n, uint32_t ok, int key0, int len) {
    const uint8_t* base = ring + slot * Gm::kStage;
    const int r = g ^ ((g >> 1) & 1);  // row order that spreads the value rows over the banks
    float S[kAdStepTiles][NT][4];
    float mx[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mx[nt][0] = mx[nt][1] = -INFINITY;
#pragma unroll
    for (int ti = 0; ti < kAdStepTiles; ++ti) {
      if (ti < n) {
        const uint8_t* tile = base + ti * Gm::kTile;
        uint32_t w0[2 * NG], w1[2 * NG], a0[NG], a1[NG];
        load_words<2 * NG>(w0, tile + r * Kv::kRow + t * (8 * NG));
        load_words<2 * NG>(w1, tile + (r + 8) * Kv::kRow + t * (8 * NG));
        load_words<NG>(a0, tile + Kv::kOffKs + r * (4 * NG));
        load_words<NG>(a1, tile + Kv::kOffKs + (r + 8) * (4 * NG));
        float acc[NT][NG][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) acc[nt][gr][0] = acc[nt][gr][1] = acc[nt][gr][2] = acc[nt][gr][3] = 0.f;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            const uint32_t x0 = w0[(s >> 1) * NG + gr], x1 = w1[(s >> 1) * NG + gr];
            const int i = 2 * (s & 1);
            const uint32_t f0 = code_pair(x0, i), f1 = code_pair(x1, i), f2 = code_pair(x0, i + 1), f3 = code_pair(x1, i + 1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_bf16(acc[nt][gr], f0, f1, f2, f3, qf[nt][gr][2 * s], qf[nt][gr][2 * s + 1]);
          }
        }
        const int key = key0 + ti * kKvTile + r;
        const bool in = (ok >> ti) & 1, v0 = in && key < len, v1 = in && key + 8 < len;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            const float c0 = sb_scale(a0[gr]) * (16.f * p.scale_log2), c1 = sb_scale(a1[gr]) * (16.f * p.scale_log2);
            const float d0 = fmaf(sb_bias(a0[gr]), p.scale_log2, -c0), d1 = fmaf(sb_bias(a1[gr]), p.scale_log2, -c1);
            s0 = fmaf(c0, acc[nt][gr][0], fmaf(d0, X[nt][gr][0], s0));
            s1 = fmaf(c0, acc[nt][gr][1], fmaf(d0, X[nt][gr][1], s1));
            s2 = fmaf(c1, acc[nt][gr][2], fmaf(d1, X[nt][gr][0], s2));
            s3 = fmaf(c1, acc[nt][gr][3], fmaf(d1, X[nt][gr][1], s3));
          }
          S[ti][nt][0] = v0 ? s0 : -INFINITY;
          S[ti][nt][1] = v0 ? s1 : -INFINITY;
          S[ti][nt][2] = v1 ? s2 : -INFINITY;
          S[ti][nt][3] = v1 ? s3 : -INFINITY;
          mx[nt][0] = fmaxf(mx[nt][0], fmaxf(S[ti][nt][0], S[ti][nt][2]));
          mx[nt][1] = fmaxf(mx[nt][1], fmaxf(S[ti][nt][1], S[ti][nt][3]));
        }
      }
    }
    // the running maximum per query and the rescaling of what was summed under the old one
    bool moved = false;
    float al[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = mx[nt][c];
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        const float now = fmaxf(m[nt][c], x);
        moved |= now > m[nt][c];
        al[nt][c] = ex2(m[nt][c] - (now == -INFINITY ? 0.f : now));
        m[nt][c] = now;
        mx[nt][c] = now == -INFINITY ? 0.f : now;  // the reference: keys that are all left out have weight 0
      }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < 2; ++c) l[nt][c] *= al[nt][c];
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          off[nt][gr][0] *= al[nt][0];
          off[nt][gr][1] *= al[nt][1];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][gr][i][e] *= al[nt][e & 1];
        }
      }
    }
#pragma unroll
    for (int ti = 0; ti < kAdStepTiles; ++ti) {
      if (ti < n) {
        const uint8_t* tile = base + ti * Gm::kTile;
        uint32_t b0[NG], b1[NG];
        load_words<NG>(b0, tile + Kv::kOffVs + r * (4 * NG));
        load_words<NG>(b1, tile + Kv::kOffVs + (r + 8) * (4 * NG));
        const int key = key0 + ti * kKvTile + r;
        const bool in = (ok >> ti) & 1, v0 = in && key < len, v1 = in && key + 8 < len;
        uint32_t f[NT][NG][2];
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          // the words of a key left out may be anything, a NaN too: as zeros they add nothing
          const uint32_t x0 = v0 ? b0[gr] : 0u, x1 = v1 ? b1[gr] : 0u;
          const float a0 = sb_scale(x0), a1 = sb_scale(x1);
          const float c0 = fmaf(8.f, a0, sb_bias(x0)), c1 = fmaf(8.f, a1, sb_bias(x1));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (gr == 0) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                S[ti][nt][e] = ex2(S[ti][nt][e] - mx[nt][e & 1]);
                l[nt][e & 1] += S[ti][nt][e];
              }
            }
            const float* P = S[ti][nt];
            const uint32_t y0 = pack_bf16(P[0] * a0, P[1] * a0), y1 = pack_bf16(P[2] * a1, P[3] * a1);
            float u0 = off[nt][gr][0], u1 = off[nt][gr][1];
            u0 = fmaf(P[0], c0, fmaf(-24.f, bf16_lo(y0), u0));
            u1 = fmaf(P[1], c0, fmaf(-24.f, bf16_hi(y0), u1));
            u0 = fmaf(P[2], c1, fmaf(-24.f, bf16_lo(y1), u0));
            u1 = fmaf(P[3], c1, fmaf(-24.f, bf16_hi(y1), u1));
            off[nt][gr][0] = u0;
            off[nt][gr][1] = u1;
            f[nt][gr][0] = movmatrix_trans(y0);
            f[nt][gr][1] = movmatrix_trans(y1);
          }
        }
        // value words of rows 2t, 2t + 1 of each half (in the row order above)
        const int r0 = (2 * t) ^ (t & 1), r1 = r0 ^ 1;
        uint32_t w0[NG], w1[NG], w2[NG], w3[NG];
        load_words<NG>(w0, tile + Kv::kOffV + r0 * Kv::kRow + g * (4 * NG));
        load_words<NG>(w1, tile + Kv::kOffV + r1 * Kv::kRow + g * (4 * NG));
        load_words<NG>(w2, tile + Kv::kOffV + (r0 + 8) * Kv::kRow + g * (4 * NG));
        load_words<NG>(w3, tile + Kv::kOffV + (r1 + 8) * Kv::kRow + g * (4 * NG));
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          // four codes of one row in the low half, the other row's in the high half
          const uint32_t x0 = __byte_perm(w0[gr], w1[gr], 0x5410), x1 = __byte_perm(w0[gr], w1[gr], 0x7632);
          const uint32_t x2 = __byte_perm(w2[gr], w3[gr], 0x5410), x3 = __byte_perm(w2[gr], w3[gr], 0x7632);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t e0 = code_pair(x0, i), e1 = code_pair(x1, i), e2 = code_pair(x2, i), e3 = code_pair(x3, i);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_bf16(o[nt][gr][i], e0, e1, e2, e3, f[nt][gr][0], f[nt][gr][1]);
          }
        }
      }
    }
  }

  template <int N>
  static __device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t* src) {
    if constexpr (N == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(src);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (N == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(src);
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(src);
    }
  }

  // lanes of one column joined; o becomes the weighted sum of the values
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int x = 4; x < 32; x *= 2) {
          l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) off[nt][gr][c] += __shfl_xor_sync(0xffffffffu, off[nt][gr][c], x);
        }
      }
#pragma unroll
      for (int gr = 0; gr < NG; ++gr)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][gr][i][e] = fmaf(16.f, o[nt][gr][i][e], off[nt][gr][e & 1]);
    }
  }

  __device__ __forceinline__ void put(float* dst) const {
    int k = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        dst[32 * k++ + lane] = m[nt][c];
        dst[32 * k++ + lane] = l[nt][c];
      }
#pragma unroll
      for (int gr = 0; gr < NG; ++gr)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[32 * k++ + lane] = o[nt][gr][i][e];
    }
  }

  __device__ __forceinline__ void add(const float* src) {
    int k = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mine[2], theirs[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float m2 = src[32 * k++ + lane], l2 = src[32 * k++ + lane];
        const float now = fmaxf(m[nt][c], m2), ref = now == -INFINITY ? 0.f : now;
        mine[c] = ex2(m[nt][c] - ref);
        theirs[c] = ex2(m2 - ref);
        l[nt][c] = l[nt][c] * mine[c] + l2 * theirs[c];
        m[nt][c] = now;
      }
#pragma unroll
      for (int gr = 0; gr < NG; ++gr)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[nt][gr][i][e] = o[nt][gr][i][e] * mine[e & 1] + src[32 * k++ + lane] * theirs[e & 1];
    }
  }

  // the block's warps into warp 0, in two rounds
  __device__ __forceinline__ void join() {
    __syncthreads();
    if (warp >= 2) put(merge + (warp - 2) * (Gm::kMerge / 4));
    __syncthreads();
    if (warp < 2) add(merge + warp * (Gm::kMerge / 4));
    __syncthreads();
    if (warp == 1) put(merge);
    __syncthreads();
    if (warp == 0) add(merge);
  }

  __device__ __forceinline__ void write_out(int seq, int hb) const {
    const int kvh = hb / p.qblocks, q0 = (hb % p.qblocks) * 8 * NT;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int qi = q0 + nt * 8 + 2 * t + c;
        if (qi >= p.group) continue;
        const float inv = l[nt][c] == 0.f ? 0.f : 1.f / l[nt][c];
        uint16_t* dst = p.out + (static_cast<long long>(seq) * p.q_heads + kvh * p.group + qi) * D + 8 * g;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          uint4 v;
          v.x = pack_bf16(o[nt][gr][0][c] * inv, o[nt][gr][1][c] * inv);
          v.y = pack_bf16(o[nt][gr][2][c] * inv, o[nt][gr][3][c] * inv);
          v.z = pack_bf16(o[nt][gr][0][c + 2] * inv, o[nt][gr][1][c + 2] * inv);
          v.w = pack_bf16(o[nt][gr][2][c + 2] * inv, o[nt][gr][3][c + 2] * inv);
          *reinterpret_cast<uint4*>(dst + 64 * gr) = v;
        }
      }
  }

  __device__ __forceinline__ void write_part(int which) const {
    const long long row0 = (static_cast<long long>(blockIdx.x) * 2 + which) * (8 * NT);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const long long row = row0 + nt * 8 + 2 * t + c;
        if (g == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * row) = make_float2(m[nt][c], l[nt][c]);
        float4* dst = reinterpret_cast<float4*>(p.part + row * D + 8 * g);
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          dst[16 * gr] = make_float4(o[nt][gr][0][c], o[nt][gr][1][c], o[nt][gr][2][c], o[nt][gr][3][c]);
          dst[16 * gr + 1] = make_float4(o[nt][gr][0][c + 2], o[nt][gr][1][c + 2], o[nt][gr][2][c + 2], o[nt][gr][3][c + 2]);
        }
      }
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(kAdThreads, 2) attn_decode_kernel(const __grid_constant__ AdParams p) {
  using Gm = AdGeom<D, NT>;
  extern __shared__ __align__(128) uint8_t ad_smem[];
  AdWarp<D, NT> W(p, ad_smem);
  const int lane = W.lane;
  if (lane == 0) {
    for (int i = 0; i < kAdStages; ++i) mbar_init(&W.bars[i], 1);
    mbar_init_fence();
  }
  __syncwarp();
  grid_launch_dependents();
  grid_dependency_wait();

  // sequences without keys, and lengths beyond their table
  for (int s = blockIdx.x; s < p.seqs; s += gridDim.x) {
    if (static_cast<long long>(__ldg(p.lens + s)) > static_cast<long long>(p.width) * p.page_tokens && threadIdx.x == 0)
      kv_error(p.err, FMOE_DEVERR_BAD_LENGTH);
    if (ad_len(p, s) == 0)
      for (int i = threadIdx.x; i < p.q_heads * (D / 8); i += kAdThreads)
        reinterpret_cast<uint4*>(p.out + static_cast<long long>(s) * p.q_heads * D)[i] = make_uint4(0u, 0u, 0u, 0u);
  }

  // the block's range of the line of units (every warp finds it for itself)
  long long total = 0;
  for (int s = lane; s < p.seqs; s += 32) total += (ad_len(p, s) + kAdStep - 1) / kAdStep;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) total += __shfl_xor_sync(0xffffffffu, total, x);
  total *= W.hbs;
  const long long blocks = min(static_cast<long long>(gridDim.x), total);
  const long long bid = blockIdx.x;
  if (threadIdx.x == 0) p.rec[bid].first = -1;
  if (bid >= blocks) return;
  const long long u0 = total * bid / blocks, u1 = total * (bid + 1) / blocks;
  AdCursor cur;
  cur.left = u1 - u0;
  long long base = 0;  // units before the sequences of this round
  for (int s0 = 0;; s0 += 32) {
    const int len = s0 + lane < p.seqs ? ad_len(p, s0 + lane) : 0;
    const long long mine = static_cast<long long>((len + kAdStep - 1) / kAdStep) * W.hbs;
    long long upto = mine;
#pragma unroll
    for (int x = 1; x < 32; x *= 2) {
      const long long y = __shfl_up_sync(0xffffffffu, upto, x);
      if (lane >= x) upto += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, base + upto > u0);
    if (past != 0) {
      const int who = __ffs(past) - 1;
      const long long in = u0 - (base + __shfl_sync(0xffffffffu, upto - mine, who));
      cur.seq = s0 + who;
      cur.len = __shfl_sync(0xffffffffu, len, who);
      cur.steps = (cur.len + kAdStep - 1) / kAdStep;
      cur.hb = static_cast<int>(in / cur.steps);
      cur.step = static_cast<int>(in % cur.steps);
      break;
    }
    base += __shfl_sync(0xffffffffu, upto, 31);
  }

  // the warp's copies run up to kAdStages steps ahead of its arithmetic, over the ends of
  // segments too
  AdCursor ahead = cur;
  int fs = 0, fhb = 0, flen = 0, fa = 0, fb = 0, flo = 0, fhi = 0;
  bool more = true;
  uint32_t issued = 0, done = 0, oks = 0;  // oks: 4 bits per ring slot
  auto refill = [&]() {
    while (more && issued - done < kAdStages) {
      while (flo >= fhi) {
        if (!W.next(ahead, fs, fhb, flen, fa, fb)) {
          more = false;
          return;
        }
        W.run(flen, fa, fb, flo, fhi);
      }
      const uint32_t slot = issued % kAdStages;
      const int n = min(kAdStepTiles, fhi - flo);
      oks = (oks & ~(0xFu << (4 * slot))) | (W.fetch(fs, fhb, flo, n, slot) << (4 * slot));
      flo += n;
      ++issued;
    }
  };
  refill();
  int seq, hb, len, a, b;
  bool begun_before = cur.step > 0;
  while (W.next(cur, seq, hb, len, a, b)) {
    W.start(seq, hb);
    int lo, hi;
    W.run(len, a, b, lo, hi);
    while (lo < hi) {
      const int n = min(kAdStepTiles, hi - lo);
      const uint32_t slot = done % kAdStages;
      W.wait(slot, (done / kAdStages) & 1u);
      W.step(slot, n, (oks >> (4 * slot)) & 0xFu, lo * kKvTile, len);
      __syncwarp();
      ++done;
      refill();
      lo += n;
    }
    W.finish();
    W.join();
    const bool ends = b == (len + kAdStep - 1) / kAdStep;
    if (W.warp == 0) {
      if (ends && !begun_before) {
        W.write_out(seq, hb);
      } else {
        W.write_part(ends ? 0 : 1);
      }
    }
    if (ends && begun_before && threadIdx.x == 0) {
      // the segment began in the block that holds its first unit: unit u lies in block
      // ((u + 1) blocks - 1) / total
      const long long end = u1 - cur.left;  // one past the segment's last unit
      const long long begin = end - (len + kAdStep - 1) / kAdStep;
      AdRecord r;
      r.first = static_cast<int>(((begin + 1) * blocks - 1) / total);
      r.seq = seq;
      r.head0 = (hb / p.qblocks) * p.group + (hb % p.qblocks) * 8 * NT;
      r.queries = min(8 * NT, p.group - (hb % p.qblocks) * 8 * NT);
      p.rec[bid] = r;
    }
    begun_before = false;
  }
}

// Joins the segments of a (sequence, head) that blocks first .. b hold: block (b, query).
// Warps take every fourth part, a lane D/32 channels.
constexpr int kAjWarps = 4;
template <int D, int NT>
__global__ void __launch_bounds__(kAjWarps * 32) attn_join_kernel(const __grid_constant__ AdParams p) {
  constexpr int C = D / 32;
  __shared__ float sl[kAjWarps], so[kAjWarps][D];
  grid_dependency_wait();
  grid_launch_dependents();
  const AdRecord r = p.rec[blockIdx.x];
  const int qi = blockIdx.y;
  if (r.first < 0 || qi >= r.queries) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int last = blockIdx.x;
  auto row = [&](int b) { return (static_cast<long long>(b) * 2 + (b == last ? 0 : 1)) * (8 * NT) + qi; };
  // the maximum over the parts, then the weighted sums
  float m = -INFINITY;
  for (int b = r.first + lane; b <= last; b += 32) m = fmaxf(m, p.part_ml[2 * row(b)]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f, o[C];
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = 0.f;
#pragma unroll 4
  for (int b = r.first + warp; b <= last; b += kAjWarps) {
    const long long at = row(b);
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
    const float w = ex2(ml.x - ref);
    l = fmaf(w, ml.y, l);
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = fmaf(w, p.part[at * D + 32 * c + lane], o[c]);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) so[warp][32 * c + lane] = o[c];
  if (lane == 0) sl[warp] = l;
  __syncthreads();
  const int ch = threadIdx.x;
  if (ch >= D) return;
  float L = 0.f, v = 0.f;
#pragma unroll
  for (int w = 0; w < kAjWarps; ++w) {
    L += sl[w];
    v += so[w][ch];
  }
  const __nv_bfloat16 y = __float2bfloat16_rn(L == 0.f ? 0.f : v * (1.f / L));
  p.out[(static_cast<long long>(r.seq) * p.q_heads + r.head0 + qi) * D + ch] = *reinterpret_cast<const uint16_t*>(&y);
}

}  // namespace fmoe
