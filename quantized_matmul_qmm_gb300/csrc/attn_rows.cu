// Attention of a step's new tokens (a drafted tree, one token, or a causal
// chunk) over a paged cache, for few query rows per key head.
//
//   s_j = scale * q . k_j,  o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m)
// over the visible j: every cached token before the step, and the new tokens
// that the row's mask (or the chain) names.  One pass over the cache with a
// running maximum and sum in fp32 (the exponentials in base 2).
//
// Decoding has one operation per row and cached byte at bf16 (4 D operations, 4 D
// bytes per token), so for the up to 16 rows that come here the cache's bytes are
// all that costs.  The kernel is a stream: four
// warps per block, each with its own ring of 16-token groups (cp.async, no
// block barrier inside an item), two blocks per SM; a group's rows are
// multiplied with mma.sync (16 x 8 x 16, bf16 with fp32 sums) straight from
// the ring.  The warps' running values are joined at the end of an item in
// shared memory, and items cut between blocks by the combine kernel.
//
// Operand layouts.  The order of the head's dimensions inside a product is
// free as long as q and k agree: a thread of the quad takes 16-byte pieces
// 4 i + c of a key row, which are its B fragments as they lie (bf16: two
// steps of 16 per piece; int8: four), and the query fragments are gathered
// to match, once per item.  bf16 values go through ldmatrix.trans; int8
// values are read as 16-byte pieces of four tokens and interleaved by byte
// permutes.  int8 codes become bf16 exactly; a token's key scale multiplies
// its column of s, its value scale the weight.  A weight meets v as two bf16
// terms (within 2^-16 of itself): one term alone would be 2^-8 off, as much as
// the output's own rounding, and the second product is free under the loads.
// The sums are fp32.
//
// Measured, heads of 128: one token of 64 requests at 3 to 8191 cached tokens,
// bf16, 173 us for 1.08 GB (0.92 of a copy's rate), fp32 queries 1 % more, int8
// 154 us for 0.54 GB (0.52); one token at 400k tokens and 8 key heads, bf16 252 us
// (0.96), int8 222 us (0.56: half the bytes, and more instructions per byte than
// issue slots); one token at 777, 8 to 9 us: the chains of loads of two launches.
// Heads of 64: 64 requests 119 us for 0.52 GB (0.65, the same steps for half the
// bytes).
//
// More rows come here where pages or scales do not allow the tile kernel's boxes
// (attn_pages_tile), in items of 32 rows, each of which reads the cache again: 32
// rows over 200k tokens, pages of 20, 180 us (pages of 16 and tiles 173), int8 190
// (163); 128 rows over 50k 181 us (54); chunks of 300 to 512 tokens 425 us (64).
// Pages that are a multiple of 8 avoid it.
//
// Rows of the cache past a request's length are never read (cp.async writes
// zeros in their place).  A new token's value row is read by all query rows
// of the tile, also by those whose mask hides it, and 0 * inf would not be 0:
// non-finite values among the new tokens are taken out of the ring, and added
// at the end to the rows that do see them.
#include <algorithm>
#include <type_traits>

#include "attn_work.cuh"
#include "umma.cuh"

namespace qmm {
namespace {

using namespace umma;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kGroup = 16;                       // cached tokens per warp step
constexpr int kTileTokens = kGroup * kWarps;     // a unit
constexpr int kBlocksPerSm = 2;
// int8 with 16 rows: three blocks.  Its loads are half as long and its
// instructions more, so that the stream waits for issue slots, not bytes (400k
// tokens: two blocks 268 us, three 250).
constexpr int blocks_per_sm(bool s8, int mt) { return s8 && mt == 1 ? 3 : kBlocksPerSm; }
constexpr int kRingBytes = 24576;                // per warp
constexpr int kCombineMaxOwners = 512;           // blocks of an attention grid, at most
// More query rows per key head than this go to the tile kernel (attn_tiles.cu).
// 400k tokens, 8 key heads, pages of 16, this kernel and the tiles: 8 to 16 rows
// bf16 260 and 323 us, int8 231 to 250 and 304; 32 rows bf16 358 and 324 (pages
// of 64: 260), int8 401 and 304.
constexpr int64_t kRowsKernelMax = 16;

template <int D, bool kS8, int MT>
struct Geo {
  static constexpr int kRow = D * (kS8 ? 1 : 2);             // bytes of a row
  static constexpr int kPieces = kRow / 16;                  // 16-byte pieces of a row
  static constexpr int kSide = kGroup * kRow;                // K or V of a group
  static constexpr int kStage = 2 * kSide + (kS8 ? 2 * kGroup * 4 : 0);
  static constexpr int kRingMax = kRingBytes * kBlocksPerSm / blocks_per_sm(kS8, MT);
  static constexpr int kStages = kRingMax / kStage < 8 ? kRingMax / kStage : 8;
  static constexpr int kRing = kStages * kStage;
  // Place of piece p of key row t: a quarter warp reads 4 pieces of 2 rows.
  QMM_DEV static uint32_t k_at(int t, int p) {
    if constexpr (kPieces >= 8) return t * kRow + ((p ^ ((t & 1) << 2)) << 4);
    else return t * kRow + (p << 4);                         // 64-byte rows: two rows fill the banks
  }
  // Place of piece p of value row t.  bf16: ldmatrix reads one piece of 8
  // rows; int8: 8 lanes read 2 pieces of the rows 2c (64-byte rows: pieces of
  // the 128-byte line that holds two rows).
  QMM_DEV static uint32_t v_at(int t, int p) {
    if constexpr (!kS8) return t * kRow + ((p ^ (t & 7)) << 4);
    else if constexpr (kPieces == 8) return t * kRow + ((p ^ (((t >> 1) & 3) << 1)) << 4);
    else return (t >> 1) * 128 + (((((t & 1) << 2) | p) ^ (((t >> 1) & 3) << 1)) << 4);
  }
};

QMM_DEV void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

QMM_DEV void ldsm_x4_trans(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr)
               : "memory");
}

QMM_DEV uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

template <int D, bool kS8, bool kQF32, int MT>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(kS8, MT))
attn_rows_kernel(const __grid_constant__ AttnArgs a) {
  using G = Geo<D, kS8, MT>;
  constexpr int kRows = 16 * MT;
  // setup: 64 requests of 3 to 8191 tokens take 185.5 us without, 178.5 with 1 unit, 174 with 2, 3 or 4
  constexpr AttnShape kShape{kRows, kTileTokens, 2};
  constexpr int kSteps = D / 16;                 // mma steps over the head's dimensions
  constexpr int kTiles = D / 8;                  // 8-column tiles of the output
  constexpr int kPitch = D + 8;                  // fp32 per row of the joining buffer
  extern __shared__ uint8_t smem_raw[];
  __shared__ AttnFindScratch find;
  __shared__ float s_ml[2][kWarps][kRows];
  __shared__ int s_bad;
  uint8_t* smem = smem_align(smem_raw, 128);
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(smem) + wid * G::kRing;
  float* joined = reinterpret_cast<float*>(smem);   // [kWarps][kRows][kPitch], after the ring is drained

  pdl_launch_dependents();
  pdl_wait();
  AttnWork w;
  if (!attn_find_work<kThreads>(a, kShape, &find, w)) {
    if (threadIdx.x == 0) attn_post_owned(a, AttnOwned{});
    return;
  }
  AttnOwned owned{};                             // the item that this block begins and another ends
  AttnWalk walk;
  walk.start(w);
  AttnItem im;
  while (walk.next(a, w, kShape, im)) {
    const AttnReq& rq = im.q;
    const int h = im.h, row0 = im.row0, kv0 = im.kv0, seg = im.seg, L = rq.L, len = im.len, n_rows = im.n_rows;
    if (im.pieces > 0) owned = attn_owned(im);
    const int tok_first = kv0 * kTileTokens + wid * kGroup;

    // ---- the ring ----
    const int32_t* trow = a.table + (int64_t)im.r * a.ld_table;
    const bool one_page = a.cache.page_size % kGroup == 0;   // a group of 16 tokens never crosses a page
    const uint8_t* kbase = a.cache.k + h * a.cache.st_head;
    const uint8_t* vbase = a.cache.v + h * a.cache.st_head;
    auto page_of = [&](int it) -> int32_t {      // of this lane's token of step it, -1 past the end
      const int tok = tok_first + it * kTileTokens + (lane & 15);
      return it < seg && tok < len ? trow[(uint32_t)tok / a.cache.page_size] : -1;
    };
    auto issue = [&](int it, int32_t page) {
      const int tok = tok_first + it * kTileTokens + (lane & 15);
      const bool live = it < seg && tok < len;
      const int64_t at = live ? attn_row_offset(a, page, tok) : -1;
      if (live && at < 0) set_status(a.dev_status, QMM_ERR_INVALID_ARG);
      const uint32_t dst = ring + (it % G::kStages) * G::kStage;
      if (it < seg) {
        constexpr int kRowsPer = 32 / G::kPieces;
        const int p = lane % G::kPieces, t_lane = lane / G::kPieces;
        if (one_page) {                          // the group's rows lie at one stride
          const int64_t first = __shfl_sync(0xffffffffu, at, 0);
          const int left = first >= 0 ? len - (tok_first + it * kTileTokens) : 0;
          const uint8_t* k = kbase + (first >= 0 ? first : 0) + t_lane * a.cache.st_token + p * 16;
          const uint8_t* v = vbase + (k - kbase);
#pragma unroll
          for (int i = 0; i < kGroup / kRowsPer; ++i) {
            const int t = t_lane + i * kRowsPer;
            const uint32_t bytes = t < left ? 16u : 0u;   // 0: nothing is read
            cp_async16_zfill(dst + G::k_at(t, p), k, bytes);
            cp_async16_zfill(dst + G::kSide + G::v_at(t, p), v, bytes);
            k += kRowsPer * a.cache.st_token;
            v += kRowsPer * a.cache.st_token;
          }
        } else {
#pragma unroll
          for (int i = 0; i < kGroup / kRowsPer; ++i) {
            const int t = t_lane + i * kRowsPer;
            const int64_t ro = __shfl_sync(0xffffffffu, at, t);
            const uint32_t bytes = ro >= 0 ? 16u : 0u;
            const int64_t src = ro >= 0 ? ro + p * 16 : 0;
            cp_async16_zfill(dst + G::k_at(t, p), kbase + src, bytes);
            cp_async16_zfill(dst + G::kSide + G::v_at(t, p), vbase + src, bytes);
          }
        }
        if constexpr (kS8) {                     // lanes 0..15: key scales, 16..31: value scales
          const float* sc = lane < 16 ? a.cache.k_scale : a.cache.v_scale;
          const uint32_t bytes = at >= 0 ? 4u : 0u;
          if (at >= 0)
            sc += ((int64_t)page * a.cache.n_heads + h) * a.cache.page_size + (uint32_t)tok % a.cache.page_size;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + 2 * G::kSide + lane * 4), "l"(sc),
                       "r"(bytes)
                       : "memory");
        }
      }
      cp_async_commit();
    };
    {
      int32_t pages[G::kStages];
#pragma unroll
      for (int s = 0; s < G::kStages; ++s) pages[s] = page_of(s);
#pragma unroll
      for (int s = 0; s < G::kStages; ++s) issue(s, pages[s]);
    }

    // ---- the query rows, as A fragments in the order of the key's pieces ----
    // int8, up to 8 rows: they stand in rows 8..15 again, whose weights are the
    // low parts, so that the products with those cost no instructions of their own
    const bool fold = kS8 && MT == 1 && n_rows <= 8;
    uint32_t qf[MT][kSteps][4];
    int node[MT][2];                             // the new token of each of the thread's rows, -1: no row
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int rr = fold ? g : mt * 16 + hf * 8 + g;
        const bool live = rr < n_rows;
        const int row = row0 + rr, i = row / a.group;
        node[mt][hf] = live ? i : -1;
        const int64_t qo = attn_q_row(a, rq, h, row);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const int d = kS8 ? 16 * c + 64 * (s >> 2) + 4 * (s & 3) : 8 * c + 32 * (s >> 1) + 4 * (s & 1);
          uint2 v = make_uint2(0, 0);
          if (live) {
            if constexpr (kQF32) {
              const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + qo + d);
              v = make_uint2(bf16_pair(f.x, f.y), bf16_pair(f.z, f.w));
            } else {
              v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.q) + qo + d);
            }
          }
          // int8 codes leave a word in the order 0, 2, 1, 3, which needs no byte permutes
          if constexpr (kS8) v = make_uint2(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632));
          qf[mt][s][hf] = v.x;
          qf[mt][s][2 + hf] = v.y;
        }
      }
    }

    float o[MT][kTiles][4];
    float m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][j][e] = 0.f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
    }
    bool bad = false;

    for (int it = 0; it < seg; ++it) {
      const int32_t next_page = page_of(it + G::kStages);
      cp_async_wait<G::kStages - 1>();
      __syncwarp();
      const int tok0 = tok_first + it * kTileTokens;
      if (tok0 < len) {
        const uint32_t kst = ring + (it % G::kStages) * G::kStage, vst = kst + G::kSide;
        float ks[2][2] = {}, vs[2][2] = {};
        if constexpr (kS8) {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const uint2 k2 = lds64(kst + 2 * G::kSide + (8 * nt + 2 * c) * 4);
            const uint2 v2 = lds64(kst + 2 * G::kSide + 64 + (8 * nt + 2 * c) * 4);
            ks[nt][0] = __uint_as_float(k2.x) * a.scale_log2, ks[nt][1] = __uint_as_float(k2.y) * a.scale_log2;
            vs[nt][0] = __uint_as_float(v2.x), vs[nt][1] = __uint_as_float(v2.y);
          }
        }
        // s = q k^T
        float s[MT][2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
#pragma unroll
          for (int i = 0; i < G::kPieces / 4; ++i) {
            const uint4 kk = lds128(kst + G::k_at(8 * nt + g, 4 * i + c));
            if constexpr (kS8) {
#pragma unroll
              for (int q4 = 0; q4 < 4; ++q4) {
                const uint32_t word = u4_get(kk, q4);
                const uint32_t b0 = s8_lanes_to_bf16(word), b1 = s8_lanes_to_bf16(word >> 8);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) mma_bf16(s[mt][nt], qf[mt][4 * i + q4], b0, b1);
              }
            } else {
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma_bf16(s[mt][nt], qf[mt][2 * i], kk.x, kk.y);
                mma_bf16(s[mt][nt], qf[mt][2 * i + 1], kk.z, kk.w);
              }
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][nt][e] *= kS8 ? ks[nt][e & 1] : a.scale_log2;
        }
        const bool masked = tok0 + kGroup > L;   // the group holds new tokens, or ends the request
        uint32_t seen[MT];                       // bit nt * 4 + e
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) seen[mt] = 0xFFu;
        if (masked) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            seen[mt] = 0;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int tok = tok0 + 8 * nt + 2 * c + (e & 1), i = node[mt][e >> 1];
                const bool v = tok < L || (tok < len && i >= 0 && attn_sees(a, rq.first, i, tok - L));
                if (v) seen[mt] |= 1u << (nt * 4 + e);
                else s[mt][nt][e] = -INFINITY;
              }
          }
          if constexpr (!kS8) {
            // non-finite values of new tokens: zeros in the ring
            bool found = false;
            for (int q16 = lane; q16 < kGroup * G::kPieces; q16 += 32) {
              const int t = q16 / G::kPieces;
              if (tok0 + t < L || tok0 + t >= len) continue;
              const uint32_t at = vst + G::v_at(t, q16 % G::kPieces);
              uint4 v = lds128(at);
              const bool hit = bf16_drop_nonfinite(v);
              if (hit) sts128(at, v);
              found |= hit;
            }
            bad |= __any_sync(0xffffffffu, found);   // also orders the stores before the loads below
            __syncwarp();
          }
        }
        // running maximum and sum, and the weights as A fragments
        uint32_t pf[MT][4], pl[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float mx = fmaxf(fmaxf(s[mt][0][2 * hf], s[mt][0][2 * hf + 1]),
                             fmaxf(s[mt][1][2 * hf], s[mt][1][2 * hf + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float m_new = fmaxf(m[mt][hf], mx);
            const float m_use = m_new == -INFINITY ? 0.f : m_new;
            if (__any_sync(0xffffffffu, m_new > m[mt][hf])) {
              const float f = exp2_approx(m[mt][hf] - m_use);
              l[mt][hf] *= f;
#pragma unroll
              for (int j = 0; j < kTiles; ++j) o[mt][j][2 * hf] *= f, o[mt][j][2 * hf + 1] *= f;
            }
            m[mt][hf] = m_new;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              float p0 = exp2_approx(s[mt][nt][2 * hf] - m_use), p1 = exp2_approx(s[mt][nt][2 * hf + 1] - m_use);
              l[mt][hf] += p0 + p1;
              if constexpr (kS8) {
                // a hidden token's scale may not be a number
                p0 = (seen[mt] >> (nt * 4 + 2 * hf)) & 1 ? p0 * vs[nt][0] : 0.f;
                p1 = (seen[mt] >> (nt * 4 + 2 * hf + 1)) & 1 ? p1 * vs[nt][1] : 0.f;
              }
              const uint32_t hi = bf16_pair(p0, p1);
              pl[mt][2 * nt + hf] = bf16_pair(p0 - bf16lo_to_f32(hi), p1 - bf16hi_to_f32(hi));
              pf[mt][2 * nt + hf] = fold && hf == 1 ? pl[mt][2 * nt + hf] : hi;
            }
          }
        }
        // o += p v
        if constexpr (!kS8) {
          const int vt = (lane & 7) + (lane & 8), vp = lane >> 4;
#pragma unroll
          for (int j = 0; j < kTiles / 2; ++j) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4_trans(vst + G::v_at(vt, 2 * j + vp), b0, b1, b2, b3);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma_bf16(o[mt][2 * j], pf[mt], b0, b1);
              mma_bf16(o[mt][2 * j + 1], pf[mt], b2, b3);
              mma_bf16(o[mt][2 * j], pl[mt], b0, b1);
              mma_bf16(o[mt][2 * j + 1], pl[mt], b2, b3);
            }
          }
        } else {
          // this thread's d of output tile j is (D / 8) g + j: tokens 2c, 2c+1, 2c+8, 2c+9
          constexpr int kWords = D / 32;         // 32-bit words of its D / 8 codes of a token
          uint32_t x[4][kWords];
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            const int t = 2 * c + (q4 & 1) + (q4 >> 1) * 8;
            if constexpr (kWords == 4) {
              const uint4 v = lds128(vst + G::v_at(t, g));
              x[q4][0] = v.x, x[q4][1] = v.y, x[q4][2] = v.z, x[q4][3] = v.w;
            } else {
              const uint2 v = lds64(vst + G::v_at(t, g >> 1) + (g & 1) * 8);
              x[q4][0] = v.x, x[q4][1] = v.y;
            }
          }
#pragma unroll
          for (int q = 0; q < kWords; ++q) {
            // [A0 A1 B0 B1], [A2 A3 B2 B3] of tokens A and B: the odd ones one byte up
            const uint32_t a01 = __byte_perm(x[0][q], x[1][q], 0x5410), a23 = __byte_perm(x[0][q], x[1][q], 0x7632);
            const uint32_t b01 = __byte_perm(x[2][q], x[3][q], 0x5410), b23 = __byte_perm(x[2][q], x[3][q], 0x7632);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t aw = e < 2 ? a01 : a23, bw = e < 2 ? b01 : b23;
              const uint32_t b0 = s8_lanes_to_bf16(e & 1 ? aw >> 8 : aw), b1 = s8_lanes_to_bf16(e & 1 ? bw >> 8 : bw);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma_bf16(o[mt][4 * q + e], pf[mt], b0, b1);
                if (!fold) mma_bf16(o[mt][4 * q + e], pl[mt], b0, b1);
              }
            }
          }
        }
      }
      __syncwarp();                              // every lane is done with the stage
      issue(it + G::kStages, next_page);
    }

    // ---- join the four warps ----
    cp_async_wait<0>();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        l[mt][hf] += __shfl_xor_sync(0xffffffffu, l[mt][hf], 1);
        l[mt][hf] += __shfl_xor_sync(0xffffffffu, l[mt][hf], 2);
        if (c == 0) {
          s_ml[0][wid][mt * 16 + hf * 8 + g] = m[mt][hf];
          s_ml[1][wid][mt * 16 + hf * 8 + g] = l[mt][hf];
        }
      }
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();                             // the ring is drained: its memory joins the outputs
    if (bad && lane == 0) s_bad = 1;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int rr = mt * 16 + hf * 8 + g;
        float top = s_ml[0][0][rr];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) top = fmaxf(top, s_ml[0][i][rr]);
        const float f = m[mt][hf] == -INFINITY ? 0.f : exp2_approx(m[mt][hf] - top);
        float* dst = joined + (wid * kRows + rr) * kPitch;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          const float x0 = o[mt][j][2 * hf] * f, x1 = o[mt][j][2 * hf + 1] * f;
          if constexpr (kS8) {                   // columns 2c and 2c + 1 of tile j are d = (D / 8) (2c) + j, ...
            dst[kTiles * (2 * c) + j] = x0;
            dst[kTiles * (2 * c + 1) + j] = x1;
          } else {
            *reinterpret_cast<float2*>(dst + 8 * j + 2 * c) = make_float2(x0, x1);
          }
        }
      }
    __syncthreads();
    const int64_t slot = 2 * (int64_t)blockIdx.x + (kv0 > 0 ? 0 : 1);
    constexpr int kLanes = D / 4;                // threads per row, four values each
    for (int rr = threadIdx.x / kLanes; rr < n_rows; rr += kThreads / kLanes) {
      const int d = (threadIdx.x % kLanes) * 4;
      float top = s_ml[0][0][rr], sum = 0.f;
#pragma unroll
      for (int i = 1; i < kWarps; ++i) top = fmaxf(top, s_ml[0][i][rr]);
      float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float mi = s_ml[0][i][rr];
        sum += s_ml[1][i][rr] * (mi == -INFINITY ? 0.f : exp2_approx(mi - top));
        const float4 v = *reinterpret_cast<const float4*>(joined + (i * kRows + rr) * kPitch + d);
        x[0] += v.x, x[1] += v.y, x[2] += v.z, x[3] += v.w;
        if (fold) {
          const float4 w = *reinterpret_cast<const float4*>(joined + (i * kRows + rr + 8) * kPitch + d);
          x[0] += w.x, x[1] += w.y, x[2] += w.z, x[3] += w.w;
        }
      }
      if (!kS8 && s_bad) attn_add_nonfinite(a, im, kTileTokens, (row0 + rr) / a.group, d, x);
      if (im.whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;   // no visible token: 0
        *reinterpret_cast<uint2*>(attn_out_row(a, rq.first, h, row0 + rr) + d) =
            make_uint2(bf16_pair(x[0] * inv, x[1] * inv), bf16_pair(x[2] * inv, x[3] * inv));
      } else {
        *reinterpret_cast<float4*>(a.part_o + (slot * kRows + rr) * D + d) = make_float4(x[0], x[1], x[2], x[3]);
        if (d == 0) a.part_ml[slot * kRows + rr] = make_float2(top, sum);
      }
    }
    __syncthreads();                             // the buffer is the next item's ring
  }
  if (threadIdx.x == 0) attn_post_owned(a, owned);
}

// Joins the pieces of the items that several blocks computed: piece 0 is the
// owner block's slot 1, the others the following blocks' slot 0.  Each block
// adds up all owners' rows and its warps take rows at the grid's pitch, so that
// a few long items keep the whole GPU busy; a warp holds the pieces' maxima and
// sums, one per lane, and four (two) columns of them per lane, eight pieces at
// a time.  What costs is the chain of loads, 3 to 4 us however little there is
// to join: the owners, then maxima, sums and the first eight pieces together.
constexpr int kCombineThreads = 256;
constexpr int kCombineWarps = kCombineThreads / 32;
constexpr int kCombinePerSm = 4;
// The owners and the running sums of their rows, in shared memory; returns the total.
struct CombineOwners {
  int end[kCombineMaxOwners];        // running sum of the owners' rows
  int4 own[kCombineMaxOwners];       // h, row0, pieces, first
  int warp[kCombineWarps];
  // the first owner whose running sum passes row i
  QMM_DEV int of(int i) const {
    int lo = 0, hi = kCombineMaxOwners - 1;
#pragma unroll 1
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (end[mid] > i) hi = mid; else lo = mid + 1;
    }
    return lo;
  }
};
QMM_DEV int combine_owners(const AttnArgs& a, CombineOwners& o) {
  constexpr int kPer = kCombineMaxOwners / kCombineThreads;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int rows[kPer], incl = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int b = threadIdx.x * kPer + k;
    rows[k] = b < a.grid ? a.owned_rows[b] : 0;
    o.own[b] = b < a.grid ? a.owned[b] : make_int4(0, 0, 0, 0);   // without rows: not looked at
    incl += rows[k];
  }
  const int mine = incl;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += up;
  }
  if (lane == 31) o.warp[wid] = incl;
  __syncthreads();
  int run = incl - mine, total = 0;
#pragma unroll
  for (int i = 0; i < kCombineWarps; ++i) {
    if (i < wid) run += o.warp[i];
    total += o.warp[i];
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) o.end[threadIdx.x * kPer + k] = run += rows[k];
  __syncthreads();
  return total;
}

template <int D>
__global__ void __launch_bounds__(kCombineThreads, kCombinePerSm)
attn_combine_kernel(const __grid_constant__ AttnArgs a, int rows_per_tile) {
  __shared__ CombineOwners s;
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kV = D / 32;                     // columns per lane
  using Vec = typename std::conditional<kV == 4, float4, float2>::type;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int total = combine_owners(a, s);
#pragma unroll 1
  for (int i = wid * gridDim.x + blockIdx.x; i < total; i += gridDim.x * kCombineWarps) {
    const int b = s.of(i), rr = i - (b > 0 ? s.end[b - 1] : 0);
    const int4 own = s.own[b];
    const int pieces = own.z;
    auto at = [&](int p) { return (int64_t)(p == 0 ? 2 * b + 1 : 2 * (b + p)) * rows_per_tile + rr; };
    Vec v[8];
    auto fetch = [&](int p0) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (p0 + k < pieces) v[k] = *reinterpret_cast<const Vec*>(a.part_o + at(p0 + k) * D + lane * kV);
    };
    fetch(0);
    const float2 ml0 = lane < pieces ? a.part_ml[at(lane)] : make_float2(-INFINITY, 0.f);
    float top = ml0.x;
#pragma unroll 1
    for (int p = 32 + lane; p < pieces; p += 32) top = fmaxf(top, a.part_ml[at(p)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float x[kV] = {}, sum = 0.f, f = 0.f;
#pragma unroll 1
    for (int p0 = 0; p0 < pieces; p0 += 8) {
      if ((p0 & 31) == 0) {                      // the next 32 pieces' factors
        const float2 ml = p0 == 0 ? ml0 : p0 + lane < pieces ? a.part_ml[at(p0 + lane)] : make_float2(-INFINITY, 0.f);
        // a piece without a maximum has no weight, unless its scores were not numbers
        f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : exp2_approx(ml.x - top);
        sum += ml.y * f;
      }
      if (p0 > 0) fetch(p0);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float fp = __shfl_sync(0xffffffffu, f, (p0 + k) & 31);
        if (p0 + k < pieces) {
          const float* e = reinterpret_cast<const float*>(&v[k]);
#pragma unroll
          for (int j = 0; j < kV; ++j) x[j] = fmaf(e[j], fp, x[j]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    __nv_bfloat16* out = attn_out_row(a, own.w, own.x, own.y + rr) + lane * kV;
    if constexpr (kV == 4)
      *reinterpret_cast<uint2*>(out) = make_uint2(bf16_pair(x[0] * inv, x[1] * inv), bf16_pair(x[2] * inv, x[3] * inv));
    else
      *reinterpret_cast<uint32_t*>(out) = bf16_pair(x[0] * inv, x[1] * inv);
  }
}

// The same with a block per row, whose warps each join a part of the row's pieces;
// the parts are then joined as pieces in their turn.  For calls of few rows, which
// may have many pieces (up to one per block of the attention kernel): one token of
// 8 query heads on one key head at 400k tokens takes 46 us (a warp per row 71), of
// 32 on 8 at 30k 29.3 (32.4); 512 rows of few pieces are better off with a warp
// each (18.8 us, here 19.8).
constexpr int kCombineRowsPerSm = 2;
template <int D>
__global__ void __launch_bounds__(kCombineThreads)
attn_combine_row_kernel(const __grid_constant__ AttnArgs a, int rows_per_tile) {
  __shared__ CombineOwners s;
  __shared__ __align__(16) float s_x[kCombineWarps][D];
  __shared__ float2 s_ml[kCombineWarps];
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kV = D / 32;
  using Vec = typename std::conditional<kV == 4, float4, float2>::type;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  if ((int)blockIdx.x >= combine_owners(a, s)) return;
  const int b = s.of(blockIdx.x), rr = blockIdx.x - (b > 0 ? s.end[b - 1] : 0);
  const int4 own = s.own[b];
  const int share = (own.z + kCombineWarps - 1) / kCombineWarps, lo = wid * share, hi = min(own.z, lo + share);
  const int64_t slot = 2 * (int64_t)b * rows_per_tile + rr;
  auto at = [&](int p) { return slot + (2 * p + (p == 0)) * rows_per_tile; };
  // a piece without a maximum has no weight, unless its scores were not numbers
  auto factor = [](float2 ml, float top) {
    return ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : exp2_approx(ml.x - top);
  };
  alignas(16) float x[kV] = {};
  Vec v[8];
  auto fetch = [&](int p0) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (p0 + k < hi) v[k] = *reinterpret_cast<const Vec*>(a.part_o + at(p0 + k) * D + lane * kV);
  };
  auto ml_at = [&](int p) { return p < hi ? a.part_ml[at(p)] : make_float2(-INFINITY, 0.f); };
  fetch(lo);
  const float2 ml0 = ml_at(lo + (lane & 7));     // of the first eight pieces, four times over
  float top = ml0.x, sum = 0.f;
#pragma unroll 1
  for (int p = lo + 8 + lane; p < hi; p += 32) top = fmaxf(top, a.part_ml[at(p)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll 1
  for (int p0 = lo; p0 < hi; p0 += 8) {
    const float2 ml = p0 == lo ? ml0 : ml_at(p0 + (lane & 7));
    if (p0 > lo) fetch(p0);
    const float f = factor(ml, top);
    sum += ml.y * f;                             // a lane's sum, four times over as well
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (p0 + k < hi) {
        const float fp = __shfl_sync(0xffffffffu, f, k);
        const float* e = reinterpret_cast<const float*>(&v[k]);
#pragma unroll
        for (int j = 0; j < kV; ++j) x[j] = fmaf(e[j], fp, x[j]);
      }
    }
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  *reinterpret_cast<Vec*>(&s_x[wid][lane * kV]) = *reinterpret_cast<const Vec*>(x);
  if (lane == 0) s_ml[wid] = make_float2(top, sum);
  __syncthreads();
  if (wid > 0) return;
  const float2 ml = s_ml[lane % kCombineWarps];
  top = ml.x;
#pragma unroll
  for (int o = kCombineWarps / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float f = factor(ml, top);
  sum = ml.y * f;
#pragma unroll
  for (int o = kCombineWarps / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  __nv_bfloat16* out = attn_out_row(a, own.w, own.x, own.y + rr) + lane * kV;
#pragma unroll
  for (int j = 0; j < kV; ++j) x[j] = 0.f;
#pragma unroll
  for (int w = 0; w < kCombineWarps; ++w) {
    const float fw = __shfl_sync(0xffffffffu, f, w);
#pragma unroll
    for (int j = 0; j < kV; ++j) x[j] = fmaf(s_x[w][lane * kV + j], fw, x[j]);
  }
#pragma unroll
  for (int j = 0; j < kV; j += 2)
    *reinterpret_cast<uint32_t*>(out + j) = bf16_pair(x[j] * inv, x[j + 1] * inv);
}

template <int D, bool kS8, bool kQF32, int MT>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t stream) {
  constexpr int kJoin = kWarps * 16 * MT * (D + 8) * 4;
  constexpr int kSmem = 128 + std::max(kWarps * Geo<D, kS8, MT>::kRing, kJoin);
  auto kern = attn_rows_kernel<D, kS8, kQF32, MT>;
  static std::atomic<uint64_t> set{0};
  const cudaError_t err = set_once(set, (const void*)kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (err != cudaSuccess) return err;
  return launch_pdl(kern, dim3(a.grid), dim3(kThreads), kSmem, stream, a);
}

template <int D, bool kS8>
cudaError_t launch_typed(const AttnArgs& a, int rows_per_tile, bool q_f32, cudaStream_t stream) {
  const bool one = rows_per_tile == 16;
  if (q_f32) return one ? launch_rows<D, kS8, true, 1>(a, stream) : launch_rows<D, kS8, true, 2>(a, stream);
  return one ? launch_rows<D, kS8, false, 1>(a, stream) : launch_rows<D, kS8, false, 2>(a, stream);
}

}  // namespace

cudaError_t launch_attn_rows(const AttnArgs& a, int rows_per_tile, bool q_f32, bool cache_s8, int head_dim,
                             cudaStream_t stream) {
  if (head_dim == 128)
    return cache_s8 ? launch_typed<128, true>(a, rows_per_tile, q_f32, stream)
                    : launch_typed<128, false>(a, rows_per_tile, q_f32, stream);
  return cache_s8 ? launch_typed<64, true>(a, rows_per_tile, q_f32, stream)
                  : launch_typed<64, false>(a, rows_per_tile, q_f32, stream);
}

template <int D>
static cudaError_t launch_combine(const AttnArgs& a, int rows_per_tile, cudaStream_t stream) {
  // the attention kernels' shared-memory configuration: an SM that had to
  // change it would drain first
  const int sms = attn_sm_count();
  const int64_t rows = a.T * (int64_t)a.n_q_heads;   // to join, at most
  const bool by_row = rows <= kCombineRowsPerSm * sms;
  auto kern = by_row ? attn_combine_row_kernel<D> : attn_combine_kernel<D>;
  static std::atomic<uint64_t> set[2] = {};
  const cudaError_t err = set_once(set[by_row], (const void*)kern,
                                   cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (err != cudaSuccess) return err;
  return launch_pdl(kern, dim3(by_row ? (unsigned)rows : kCombinePerSm * sms), dim3(kCombineThreads), 0, stream, a,
                    rows_per_tile);
}

cudaError_t launch_attn_combine(const AttnArgs& a, int rows_per_tile, int head_dim, cudaStream_t stream) {
  return head_dim == 128 ? launch_combine<128>(a, rows_per_tile, stream) : launch_combine<64>(a, rows_per_tile, stream);
}

// ---- the choice of a kernel, shared by the size query and the call ----

int attn_sm_count() {
  static std::atomic<int> known[64] = {};       // per device
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) != cudaSuccess) return sms;
  if (dev < 64 && known[dev].load(std::memory_order_relaxed) > 0) return known[dev].load(std::memory_order_relaxed);
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && dev < 64)
    known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

bool attn_pages_tile(const KvView& c, bool s8) {
  // TMA boxes of whole 8-row groups inside a page, strides that a tensor map
  // holds, and 16-byte loads of four scales
  constexpr int64_t kMaxStride = (int64_t)1 << 40;
  return c.page_size % 8 == 0 && c.st_page < kMaxStride && c.st_token < kMaxStride && c.st_head < kMaxStride &&
         (!s8 || (aligned(c.k_scale, 16) && aligned(c.v_scale, 16)));
}

AttnPlan attn_plan(int64_t rows, bool pages_tile, bool s8) {
  const int sms = std::min(attn_sm_count(), kCombineMaxOwners / 3);
  if (rows > kRowsKernelMax && pages_tile) return {true, rows <= 128 ? 128 : 256, sms};
  return {false, rows <= 16 ? 16 : 32, blocks_per_sm(s8, rows <= 16 ? 1 : 2) * sms};
}

namespace {
size_t plan_bytes(const AttnPlan& p, int head_dim) {
  return 2 * (size_t)p.grid * p.rows_per_tile * (head_dim * sizeof(float) + sizeof(float2)) +
         (size_t)p.grid * (sizeof(int4) + sizeof(int));
}
}  // namespace

size_t attn_workspace_bytes(int64_t rows, int head_dim) {
  size_t most = 0;                               // whatever the cache's type and pages turn out to be
  for (int i = 0; i < 4; ++i) most = std::max(most, plan_bytes(attn_plan(rows, i & 1, i & 2), head_dim));
  return most;
}

cudaError_t launch_attn(AttnArgs& a, bool q_f32, bool cache_s8, int head_dim, void* workspace, cudaStream_t stream) {
  const AttnPlan p = attn_plan((int64_t)a.max_new * a.group, attn_pages_tile(a.cache, cache_s8), cache_s8);
  a.grid = p.grid;
  const size_t rows = 2 * (size_t)p.grid * p.rows_per_tile;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + rows * head_dim);
  a.owned = reinterpret_cast<int4*>(a.part_ml + rows);
  a.owned_rows = reinterpret_cast<int*>(a.owned + p.grid);
  const cudaError_t err = p.tiles ? launch_attn_tiles(a, p.rows_per_tile, q_f32, cache_s8, head_dim, stream)
                                  : launch_attn_rows(a, p.rows_per_tile, q_f32, cache_s8, head_dim, stream);
  if (err != cudaSuccess) return err;
  return launch_attn_combine(a, p.rows_per_tile, head_dim, stream);
}

}  // namespace qmm
