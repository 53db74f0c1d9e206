// Attention of one new token per sequence over dense-layout pages: kernels, included by one
// translation unit per element type (paged_attn_f16.cu, paged_attn_bf16.cu, paged_attn_e4m3.cu).
//
//   s_p = scale q . k_p,  out = sum_p 2^(s_p log2(e) - m) v_p / sum_p 2^(s_p log2(e) - m)
//
// What bounds it: reading the cache once.  A step does 4 d operations per query head for the 4 d bytes (16
// bits) of a token's key and value, far below what the tensor cores do in that time, so everything here
// serves one aim: enough bytes in flight on every multiprocessor from the first moment to the last.
//
// Work split.  A segment is one (sequence, KV head, group of up to 8 NT query heads); its work is its
// number of pages plus kLead for the queries, the joining and the result.  All segments stand in one line, and
// T teams get equal pieces of it, whatever the lengths are: a ragged batch and a single long sequence are split
// alike, in one wave, with no length known on the host.  Cuts that fall within a segment's lead, or within kTau pages
// of its ends, move to the end.  A team is one warp: what a segment costs beside its pages (fetching its queries,
// joining, writing) is hidden by the CTA's other warps, where a team of all warps would wait for it (measured:
// 64 sequences of 0.5 to 16K tokens, e4m3, 32 / 8 heads: 3.3 us per segment and CTA).  A segment
// that one warp holds whole is written out from registers.  The pieces of a cut one are joined in shared memory when
// the CTA's warps are through, and what crosses CTAs (at most two pieces per CTA) by the merge kernel.
//
// One page (16 tokens) per warp and step, each warp with a ring of S stages that it fills itself by TMA (128-byte
// swizzle, so that the rows of a plain [16][d] tile are read without bank conflicts) and mbarriers:
//   S^T = K Q^T   mma.m16n8k16, A = 16 tokens x 16 dims of K (ldmatrix), B = 8 heads of Q in registers
//   O^T += V^T P^T            A = 16 dims x 16 tokens of V (ldmatrix.trans), B = P^T (movmatrix of S^T's layout)
// (8-bit pages: bytes are transposed by ldmatrix.m16n16.b8, its rows ordered as the weights' fragments want them.)
// With tokens and dims on the 16-row side, 8 query heads per KV head fill the 8-column side and no row of the
// products is padding; the accumulators are d / 4 registers.
//
// Precision: q and k products are exact and summed in fp32.  A weight is split into parts whose products with V are
// exact.  Each page's sum leaves the tensor core and is added to the running sum by an fp32 addition that rounds to
// nearest (the tensor core cuts, which over thousands of pages would pull the sum towards zero); the weights' total is a
// compensated sum.  The running maximum m is a whole number that is only raised when a score passes it by more
// than 8, so that most pages rescale nothing, and then by a power of two.  Weights of the total are 2^(s - m) <= 2^8, those
// of the values 2^-8 times that, at most 1: a sum of values overflows where the number of tokens times the largest
// value does.
//   16-bit pages: three bf16 parts (24 bits) beside bf16 values, two tf32 parts (22 bits) beside fp16 values, which are
// exact in tf32.  Both have the exponents of fp32: a part of a small weight is as good as one of a large one, so
// it does not matter what a token's values are worth beside its neighbours'.  (Two fp16 parts end at 2^-25, and a token
// of small weight and large values then loses its bits.)  Two fp16 parts take the same time: 16 ragged sequences
// 624 us, tf32 parts 622.
//   e4m3 pages: codes are exact in fp16, and tf32 parts would cost their widening (64 ragged sequences 186 against
// 173 us), so the weights have two fp16 parts.  Key exponents scale the fp32 scores, value exponents the weights.  As the
// exponent is the size of a token's values, weight and exponent together say what the token is worth in the result: a
// second reference per head, a power of two, holds the largest of these below 2^15 and, when it is set, at 2^12.  What
// the parts leave out is 2^-37 of the largest token's share.
//   bf16 queries on e4m3 pages are scaled by a power of two per head into fp16's range (exact down to 2^-31 of the
// head's largest entry); half of its inverse comes before a key's exponent and half behind it, so that large
// keys with small queries do not overflow on the way.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <math_constants.h>

#include "common.cuh"
#include "paged.cuh"

namespace tq {
namespace {

enum { kF16 = 0, kBF16 = 1, kE4M3 = 2 };

constexpr float kLazy = 8.f;                     // the reference is raised when a score passes it by more than this
constexpr float kDown = 1.f / 256, kUp = 256.f;  // values are summed with weights of at most 1: 2^-kLazy, and back
constexpr float kNone = -3.402823466e38f;        // m before the first score
// e4m3 pages: the values' reference is set so that the largest product is in [2^12, 2^13), and lowered when one
// passes 2^15; it begins at 2^100 and stays within 2^-113 and 2^100
constexpr int kValueAt = 12, kValueMost = 15, kValueTop = 100, kValueLeast = -113;

template <int KIND, int D, int NT>
struct PagedCfg {
  static constexpr int ES = KIND == kE4M3 ? 1 : 2;
  static constexpr int HALF = kPage * D * ES;  // keys or values of a page
  static constexpr int PAGE = 2 * HALF;
  static constexpr int EXP = KIND == kE4M3 ? 32 : 0;
  static constexpr int HEADS = 8 * NT;
  static constexpr bool QREG = D * NT <= 128;              // query fragments in registers
  static constexpr int QBYTES = QREG ? 0 : HEADS * D * 2;  // else in shared memory, per warp
  // A cut segment's sums: [HEADS][PITCH] floats (padded against bank conflicts where there is room) for the piece
  // that continues one; the piece that begins one is a warp's last, its stages are free to hold it.
  static constexpr int PITCH = D < 512 && (NT == 1 || D == 64) && !(KIND == kE4M3 && D == 128) ? D + 4 : D;
  static constexpr int SLOT = HEADS * PITCH * 4 + HEADS * 16 + 32;
  static constexpr bool LENS = D < 512;  // the lengths in shared memory (no room for them at 512)
  static constexpr int LIMIT = 232448 - 1024;  // 227 KB, less the alignment of the stages
  static constexpr int fixed(int nw) { return nw * (SLOT + QBYTES) + nw * 32 * (LENS ? 8 : 4) + nw * 4 + (nw == 16 ? nw * 48 : 0); }
  static constexpr int per(int nw) { return nw * (PAGE + EXP + 16); }
  static constexpr int stages(int nw) { return (LIMIT - fixed(nw)) / per(nw); }
  static constexpr int MIN_S = (HEADS * PITCH * 4 + PAGE - 1) / PAGE;  // a warp's stages hold its last piece
  static constexpr bool fits(int nw, int s) { return stages(nw) >= (s > MIN_S ? s : MIN_S); }
  // Warps per CTA: as many as fit.  Stages: as many whole ones as stay within 96 KB (e4m3) or 128 KB per multiprocessor,
  // which rounds down.  On the way, with up to 8 heads a segment and with 16: 16-bit pages 128 and 128 KB at d = 64, 96
  // and 64 at 128 and 256, 128 at 512; e4m3 pages 96 and 96 at d = 64, 64 and 96 at 128, 96 and 96 at 256, 64 at 512.  More
  // is not better: with every queue full the multiprocessors farther from memory fall behind and the last of
  // them ends late.  16-bit pages of d = 128, 8 x 32K and 16 ragged sequences: 12 warps x 1 stage (96 KB) 85.8 and 622 us,
  // 8 x 2 (128 KB) 87.0 and 634, 16 x 1 (128 KB) 88.7 and 644.  e4m3 pages of d = 128, 64 ragged sequences: 16 x 1 (64 KB)
  // 173 us, 16 x 2 (128 KB) 181.
  // (e4m3 at d = 64 with 16 query heads has no registers for 16 warps: 16 92.1 us, 12 87.2.)
  static constexpr int NW = PAGE <= 4096 && QREG && (NT == 1 || KIND != kE4M3) && fits(16, 1) ? 16 : fits(12, 1) ? 12 : fits(8, 1) ? 8 : fits(6, 1) ? 6 : 4;
  static constexpr int S_WANT = (KIND == kE4M3 ? 96 : 128) * 1024 / (NW * PAGE);
  static constexpr int S_LEAST = S_WANT > MIN_S ? S_WANT : MIN_S;
  static constexpr int S = S_LEAST < stages(NW) ? S_LEAST : stages(NW);
  static_assert(S >= 1 && S <= 8, "one stage per warp fits");
  static constexpr int THREADS = NW * 32;
  static_assert(HEADS * PITCH * 4 <= S * PAGE, "a warp's stages hold its last piece");
  // dynamic shared memory, from a 1024-byte aligned base
  static constexpr int OFF_SLOT = NW * S * PAGE;                    // [NW][HEADS][PITCH]
  static constexpr int OFF_ML = OFF_SLOT + NW * HEADS * PITCH * 4;  // [2][NW][HEADS] references and totals
  static constexpr int OFF_REC = OFF_ML + NW * HEADS * 16;          // [2][NW] what the pieces are
  static constexpr int OFF_Q = OFF_REC + NW * 32;
  static constexpr int OFF_EXP = OFF_Q + NW * QBYTES;
  static constexpr int OFF_BAR = OFF_EXP + NW * S * EXP;
  static constexpr int OFF_PRE = OFF_BAR + NW * S * 16;
  static constexpr int OFF_WARP = OFF_PRE + THREADS * 4;
  static constexpr int OFF_LEN = OFF_WARP + NW * 4;
  // with 16 warps (128 registers a thread) the way of the fetches is kept here between batches
  static constexpr bool PARK = NW == 16;
  static constexpr int OFF_WALK = (OFF_LEN + (LENS ? THREADS * 4 : 0) + 15) / 16 * 16;
  static constexpr int SMEM = OFF_WALK + (PARK ? NW * 48 : 0) + 1024;
  static_assert(SMEM <= 232448, "shared memory");
  static constexpr int SWIZZLE_ROW = D * ES < 128 ? D * ES : 128;  // bytes of a row in one TMA box
  static constexpr int BOXES = D * ES / SWIZZLE_ROW;               // boxes side by side in a page
  // With one stage keys and values are copied apart, so that the next keys come while the values are used (e4m3 at d = 512
  // 68.6 against 79.9 us); with more a page is one copy and one wait (fewer instructions: e4m3 at d = 64 55.9 against 64.9).
  static constexpr bool APART = S == 1;
  // The weights' total grows by every page: its rounding is the largest error of a long sequence (16 ragged sequences up
  // to 128K tokens: 1.2e-6 of the result, 4.2e-7 with what is lost kept; the same time).  8-bit pages with 16
  // heads or d = 512 go without (with it 87.5 against 85.6 us at d = 64, 74.1 against 72.9 at 128, 71.9 against 68.6 at 512).
  static constexpr bool KEEP_LOST = KIND != kE4M3 || (NT == 1 && D < 512);
  static constexpr int BOX_ROWS = APART ? kPage : 2 * kPage;
  static constexpr int BOX = BOX_ROWS * SWIZZLE_ROW;
};

// ---------------------------------------------------------------- work split, shared by both kernels
// A segment's queries, joining and result cost a warp about two pages' time: kLead units of the line beside its pages (2: 256
// short sequences 29.6 us, 64 ragged e4m3 173.2; 0: 36.0 and 174.8; 4: 30.2 and 174.0).  Pieces go down to one unit:
// more warps shorten a small call's chain (1 x 1K 10.0 us, from two units on 10.5).  Cuts within kTau pages of a
// segment's ends move there, which saves pieces of one page; more cost balance (4: 256 short 32.4, sliding window at d
// 256 31.1 against 28.7).
constexpr int kLead = 2, kTau = 1;

struct PagedPlan {
  int teams;       // most teams: the grid's warps
  int unit;        // the line counts 2^unit pages as one, so that it stays below 2^31
  int groups;      // query-head groups per KV head
  uint32_t wait_limit;  // nanoseconds that a warp waits for a copy
};

struct PagedWork {
  PagedArgs a;
  PagedPlan p;
  int q_bf16;
  int2* cuts;    // workspace: per segment the first and the last CTA with a piece of it, written by the first
  float* parts;  // workspace: per CTA the piece that comes from the CTA in front, and the one that goes on behind
};

struct Seq {
  int len, lo, first, pages;  // length, first position seen, first page, pages seen
};
__device__ __forceinline__ bool length_ok(const PagedArgs& a, int len) {
  return len >= 0 && len <= (int64_t)a.max_blocks * kPage;
}
__device__ __forceinline__ Seq seq_of(const PagedArgs& a, int len) {
  Seq s;
  s.len = length_ok(a, len) ? len : 0;
  s.lo = a.window && s.len > a.window ? s.len - a.window : 0;
  s.first = s.lo / kPage;
  s.pages = s.len ? (s.len + kPage - 1) / kPage - s.first : 0;
  return s;
}
// Length of one segment of the sequence on the line.
__device__ __forceinline__ int span_of(const PagedPlan& p, const Seq& s) {
  return s.pages ? ((s.pages + (1 << p.unit) - 1) >> p.unit) + kLead : 0;
}

// Equal pieces of the line: piece t begins at t base + min(t, rest).
struct Pieces {
  unsigned teams, rest, base;
  __device__ __forceinline__ Pieces(const PagedPlan& p, unsigned work) {
    teams = min(max(work, 1u), (unsigned)p.teams);
    base = work / teams;
    rest = work - base * teams;
  }
  __device__ __forceinline__ unsigned begin(unsigned t) const { return t * base + min(t, rest); }
  // the first piece that begins at x or behind it
  __device__ __forceinline__ unsigned from(unsigned x) const {
    const unsigned big = rest * (base + 1);
    return x <= big ? (x + base) / (base + 1) : rest + (x - big + base - 1) / base;
  }
};

// ---------------------------------------------------------------- PTX
__device__ __forceinline__ uint32_t sm_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Bounded wait, `limit` nanoseconds of %globaltimer (0: none, and no look either); false on expiry.  Lanes poll each for
// itself, so near the limit their answers can differ.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, uint32_t limit) {
  if (limit == 0) return false;
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    if (ok) return true;
    if ((i & 63) == 0) {
      uint64_t now;
      asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
      if (i == 0) t0 = now;
      else if (now - t0 > limit) return false;
    }
  }
}
constexpr uint32_t kLate = 0x80000000u;        // in a lane's word of barrier phases: it has given up waiting
constexpr uint32_t kDrainLimit = 1000000000u;  // for the copies under way when a lane has given up
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Two 16 x 16 tiles of bytes, transposed: rows g and g + 8 of the first, then of the second, bytes 4 t .. 4 t + 3.
__device__ __forceinline__ void ldsm2t8(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movmat(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool BF>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same with nothing to add to.
template <bool BF>
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// d += A B, A 16 dims x 8 tokens and B 8 tokens x 8 heads of tf32.
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// Two fp16 as the fp32 they are, which tf32 (10 fraction bits, 8 exponent bits) holds.
__device__ __forceinline__ void widen(uint32_t two, uint32_t& lo, uint32_t& hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
  lo = __float_as_uint(f.x);
  hi = __float_as_uint(f.y);
}
// 2^x; -inf gives +0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two e4m3 codes (low byte first) as two fp16.
__device__ __forceinline__ uint32_t f16_of_e4m3(uint32_t two) {
  uint32_t r;
  asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo; }" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t f16_of_e4m3_high(uint32_t four) {
  uint32_t r;
  asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, hi; }" : "=r"(r) : "r"(four));
  return r;
}
// 2^e for e in [-126, 127]; 0 for -127.
__device__ __forceinline__ float power2(int e) { return __int_as_float((e + 127) << 23); }

// The exponent of a positive normal number, as of 2^e (of an infinity 128).
__device__ __forceinline__ int exponent_in(float x) { return (__float_as_int(x) >> 23) - 127; }

// 16-bit parts of a pair of fp32 weights: each part rounds what the ones before leave.
template <bool BF>
__device__ __forceinline__ uint32_t take_part(float& x, float& y) {
  if (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
    x -= __uint_as_float(u << 16);
    y -= __uint_as_float(u & 0xffff0000u);
    return u;
  }
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  x -= f.x;
  y -= f.y;
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Weights of 8 tokens (row g) and heads 2 t, 2 t + 1 handed over as those of head g and tokens 2 t, 2 t + 1: the fp32
// words by their 16-bit halves.
__device__ __forceinline__ void turn(float& x, float& y) {
  const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
  const uint32_t h = movmat(__byte_perm(a, b, 0x7632)), l = movmat(__byte_perm(a, b, 0x5410));
  x = __uint_as_float(__byte_perm(l, h, 0x5410));
  y = __uint_as_float(__byte_perm(l, h, 0x7632));
}
// tf32 parts of an fp32 weight: the first 11 bits cut off (a NaN stays one), and what is left rounded to 11.
__device__ __forceinline__ void tf32_parts(float x, uint32_t& high, uint32_t& low) {
  high = __float_as_uint(x) & 0xffffe000u;
  low = (__float_as_uint(x - __uint_as_float(high)) + 0x1000u) & 0xffffe000u;
}

// ---------------------------------------------------------------- scan and walk over the line
struct Scan {
  const unsigned* pre;  // the line in front of each entry of `stride` sequences
  const int* len;      // the sequences' lengths in shared memory, or NULL
  int stride;
  unsigned heads;      // segments per sequence
  __device__ __forceinline__ Seq seq(const PagedArgs& a, int b) const {
    return seq_of(a, len ? len[b] : a.lengths[b]);
  }
};

// The segment at a point of the line: sequence b, segment hg of it, at `at` of its `span`.
struct At {
  int b, hg, at, span;
  Seq s;
};
// The segments at x (lanes 0..15) and y (lanes 16..31); front: the line in front of the scan's entries 32 lane.  For
// a whole warp.
__device__ __forceinline__ At locate(const PagedArgs& a, const PagedPlan& p, const Scan& sc, unsigned front, unsigned x, unsigned y,
                                     int lane) {
  // the last entries that do not begin behind x and y: first their block of 32, then in it
  const int bx = (__popc(__ballot_sync(kFull, front <= x)) - 1) * 32, by = (__popc(__ballot_sync(kFull, front <= y)) - 1) * 32;
  const int ex = bx + __popc(__ballot_sync(kFull, sc.pre[bx + lane] <= x)) - 1;
  const int ey = by + __popc(__ballot_sync(kFull, sc.pre[by + lane] <= y)) - 1;
  const int e = lane < 16 ? ex : ey;
  At r;
  unsigned at = (lane < 16 ? x : y) - sc.pre[e];
  r.b = e * sc.stride;
  for (;;) {
    r.s = sc.seq(a, r.b);
    r.span = span_of(p, r.s);
    if (sc.stride == 1 || at < r.span * sc.heads || r.b + 1 >= a.batch) break;
    at -= r.span * sc.heads;
    ++r.b;
  }
  r.hg = at / (unsigned)r.span;
  r.at = at - r.hg * r.span;
  return r;
}

// The KV head of a segment.
__device__ __forceinline__ int kv_head(const PagedPlan& p, int hg) { return p.groups == 1 ? hg : hg / p.groups; }

// Moves a cut at x, which is in segment r, to that segment's end or beginning where it is near.
__device__ __forceinline__ unsigned settle(const PagedPlan& p, const At& r, unsigned x) {
  if (r.at <= kLead + kTau) return x - r.at;
  if (r.span - r.at <= kTau) return x - r.at + r.span;
  return x;
}

// A warp's way along its piece of the line, by portions: its share of one segment, pages p .. p + take - 1.
struct __align__(16) Walk {
  int b, hg;
  int at, end, span;  // the portion is at .. end of the segment's span
  int p, take;        // its first page and its pages
  Seq s;
  int left;           // what the warp has from this portion on
  __device__ __forceinline__ void open(const PagedPlan& pl) {
    end = min(at + left, span);
    p = max(at - kLead, 0) << pl.unit;
    take = max(min((end - kLead) << pl.unit, s.pages) - p, 0);
  }
  __device__ __forceinline__ bool next(const PagedArgs& a, const PagedPlan& pl, const Scan& sc) {
    left -= end - at;
    if (left <= 0) return false;
    at = 0;
    if (++hg == (int)sc.heads) {
      hg = 0;
      do {
        if (++b >= a.batch) return false;
        s = sc.seq(a, b);
      } while (s.pages == 0);
      span = span_of(pl, s);
    }
    open(pl);
    return true;
  }
};

// ln of the weights' sum L, which is relative to 2^M
__device__ __forceinline__ float lse_of(float M, float L) {
  return L == 0.f ? -CUDART_INF_F : (M + log2f(L)) * 0.69314718055994530942f;
}
// What turns the values' sum into the result.
__device__ __forceinline__ float inverse_of(float L) { return L == 0.f ? 0.f : kUp / L; }

// ---------------------------------------------------------------- the kernel
template <int KIND, int D, int NT>
__global__ void __launch_bounds__(PagedCfg<KIND, D, NT>::THREADS, 1)
    paged_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ PagedWork w) {
  using C = PagedCfg<KIND, D, NT>;
  constexpr bool BF = KIND == kBF16, F8 = KIND == kE4M3;
  constexpr int NW = C::NW, S = C::S, KS = D / 16;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024 - (sm_addr(raw) & 1023)) & 1023);
  unsigned* pre = reinterpret_cast<unsigned*>(sm + C::OFF_PRE);
  const PagedArgs& a = w.a;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g = lane >> 2, t = lane & 3;
  const int heads = a.hkv * w.p.groups;  // segments per sequence
  const uint32_t stage0 = sm_addr(sm) + wid * S * C::PAGE, bar0 = sm_addr(sm + C::OFF_BAR) + wid * S * 16;
  const uint32_t exp0 = sm_addr(sm + C::OFF_EXP) + wid * S * C::EXP;
  float* own_stage = reinterpret_cast<float*>(sm + wid * S * C::PAGE);
  float* own_slot = reinterpret_cast<float*>(sm + C::OFF_SLOT) + wid * C::HEADS * C::PITCH;
  float2* ml = reinterpret_cast<float2*>(sm + C::OFF_ML);
  int4* rec = reinterpret_cast<int4*>(sm + C::OFF_REC);

  // what needs no input of the stream comes before the wait for the kernel in front
  asm volatile("griddepcontrol.launch_dependents;");
  if (tid == 0 && a.num_blocks > 0) asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
  if (lane < 2 * S) bar_init(bar0 + 8 * lane, 1);
  if (lane < 2) rec[lane * NW + wid] = make_int4(0, 0, 0, 0);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- scan: the line in front of each entry of `stride` sequences
  int* len_sm = reinterpret_cast<int*>(sm + C::OFF_LEN);
  Scan sc;
  sc.pre = pre;
  sc.stride = (a.batch + C::THREADS - 1) / C::THREADS;
  sc.heads = heads;
  sc.len = C::LENS && sc.stride == 1 ? len_sm : nullptr;
  unsigned own = 0;
  bool bad_len = false;
  for (int b = tid * sc.stride; b < min((tid + 1) * sc.stride, a.batch); ++b) {
    const int len = a.lengths[b];
    if (C::LENS) len_sm[tid] = len;  // used where stride is 1
    bad_len |= !length_ok(a, len);
    own += span_of(w.p, seq_of(a, len)) * heads;
  }
  unsigned inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned up = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += up;
  }
  unsigned* wsum = reinterpret_cast<unsigned*>(sm + C::OFF_WARP);
  if (lane == 31) wsum[wid] = inc;
  __syncthreads();
  unsigned front = lane < NW ? wsum[lane] : 0, work;
#pragma unroll
  for (int o = 1; o < NW; o <<= 1) {
    const unsigned up = __shfl_up_sync(kFull, front, o);
    if (lane >= o) front += up;
  }
  work = __shfl_sync(kFull, front, NW - 1);
  front = __shfl_up_sync(kFull, front, 1);  // the line in front of warp `lane`'s entries
  if (lane == 0) front = 0;
  if (lane >= NW) front = 0xffffffffu;
  pre[tid] = __shfl_sync(kFull, front, wid) + inc - own;
  if (blockIdx.x == 0 && bad_len) flag_error(a.err, TQ_DEVERR_POSITION);
  if (work == 0) return;
  const Pieces pieces(w.p, work);
  __syncthreads();

  if (blockIdx.x * NW >= pieces.teams) return;

  // ---- this warp's piece
  const unsigned team = blockIdx.x * NW + wid;
  Walk out{}, in_reg;    // the portion being computed, and the one being fetched
  unsigned x_end = 0;    // where the piece ends
  bool busy = team < pieces.teams;
  if (busy) {
    unsigned x0 = pieces.begin(team), x1 = pieces.begin(team + 1);
    At r = locate(a, w.p, sc, front, x0, min(x1, work - 1), lane);
    const unsigned x = settle(w.p, r, lane < 16 ? x0 : x1);
    const int back = __shfl_sync(kFull, r.at, 0), over = __shfl_sync(kFull, r.span, 0) - back;
    x0 = __shfl_sync(kFull, x, 0);
    x1 = __shfl_sync(kFull, x, 16);
    if (team + 1 == pieces.teams) x1 = work;
    busy = x0 < x1;
    if (busy) {
      if (back > kLead + kTau && over <= kTau) r = locate(a, w.p, sc, front, x0, x0, lane);  // the next segment
      out.b = __shfl_sync(kFull, r.b, 0);
      out.hg = __shfl_sync(kFull, r.hg, 0);
      out.at = __shfl_sync(kFull, r.at, 0);
      if (out.at <= kLead + kTau) out.at = 0;
      out.s = sc.seq(a, out.b);
      out.span = span_of(w.p, out.s);
      out.left = x1 - x0;
      out.open(w.p);
      x_end = x1;
    }
  }

  // ---- fetching
  // Block ids are looked up by batches of up to 32 pages (one per lane), a batch ahead, and the queries of a new
  // portion are brought to L1 then: with every stage in flight a load waits its turn for microseconds.
  int in_i = 0, next_n = 0, next_id = -1, next_kvh = 0;
  int cur_i = 0, cur_n = 0, tiles = -1, tile = -1;
  bool in_done = !busy;
  uint32_t valid = 0, parity = 0, vparity = 0;  // bit per stage: a page is there or on its way; phases of the barriers
  bool bad_id = false;
  // A lane whose wait runs out is late (kLate in `parity`): it waits for nothing more, and lane 0 then starts no more
  // copies, but it goes on with the warp, which computes with whatever the stages hold: lanes near the limit can differ,
  // and everything here is written for whole warps.  At the end of a portion one late lane makes the warp's rows NaN.
  Walk* parked = reinterpret_cast<Walk*>(sm + C::OFF_WALK) + wid;
  auto enter = [&](const Walk& in) {
    in_i = 0;
    next_kvh = kv_head(w.p, in.hg);
    const int h0 = (in.hg - next_kvh * w.p.groups) * C::HEADS;
    const char* q = reinterpret_cast<const char*>(a.q + in.b * a.q_stride + ((int64_t)next_kvh * a.n_rep + h0) * D);
    for (int off = lane * 128; off < min(C::HEADS, a.n_rep - h0) * D * 2; off += 32 * 128)
      asm volatile("prefetch.global.L1 [%0];" ::"l"(q + off));
  };
  auto load_batch = [&]() {
    Walk in;
    if constexpr (C::PARK) in = *parked;
    else in = in_reg;
    const bool moves = !in_done && in_i == in.take;
    while (!in_done && in_i == in.take) {
      in_done = !in.next(a, w.p, sc);
      if (!in_done) enter(in);
    }
    if constexpr (C::PARK) {
      __syncwarp();
      if (moves && lane == 0) *parked = in;
      __syncwarp();
    } else {
      in_reg = in;
    }
    next_n = in_done ? 0 : min(in.take - in_i, 32);
    if (lane < next_n) next_id = a.block_table[(int64_t)in.b * a.max_blocks + in.s.first + in.p + in_i + lane];
    in_i += next_n;
  };
  if (busy) {
    if constexpr (C::PARK) {
      if (lane == 0) *parked = out;
      __syncwarp();
    } else {
      in_reg = out;
    }
    enter(out);
    load_batch();
  }
  // Step to the next page of this warp: its tile in `tile` (-1: a bad id); false when there is none.
  auto fetch_next = [&]() -> bool {
    if (cur_i == cur_n) {
      if (next_n == 0) return false;
      cur_n = next_n;
      cur_i = 0;
      const bool ok = next_id >= 0 && next_id < a.num_blocks;
      bad_id |= lane < cur_n && !ok;
      tiles = ok ? next_id * a.hkv + next_kvh : -1;
      load_batch();
    }
    tile = __shfl_sync(kFull, tiles, cur_i);
    ++cur_i;
    return true;
  };
  // Lane 0 starts the copies of a page's keys (side 0) or values (1), or of the whole page (side 0).
  auto fetch = [&](int st, int side) {
    const uint32_t bar = bar0 + 16 * st + 8 * side, dst = stage0 + st * C::PAGE + side * C::HALF;
    bar_expect(bar, (C::APART ? C::HALF : C::PAGE) + (side == 0 ? C::EXP : 0));
#pragma unroll
    for (int j = 0; j < C::BOXES; ++j)
      tma_load(dst + j * C::BOX, &map, j * (C::SWIZZLE_ROW / C::ES), side * kPage, tile, bar);
    if (F8 && side == 0)
      bulk_load(exp0 + st * C::EXP, a.pool + (size_t)tile * (C::PAGE + C::EXP) + C::PAGE, C::EXP, bar);
  };
  // Before a late lane 0 goes on, the copies that it has on their way come to their end: a phase of each barrier at most is
  // open, the keys' of the stages in `valid`, the values' of those in `values`.  The other lanes started none.
  auto give_up = [&](uint32_t values) {
    parity |= kLate;
#pragma unroll 1
    for (int k = 0; k < S && lane == 0; ++k) {
      if (valid >> k & 1) bar_wait(bar0 + 16 * k, parity >> k & 1, kDrainLimit);
      if (C::APART && (values >> k & 1)) bar_wait(bar0 + 16 * k + 8, vparity >> k & 1, kDrainLimit);
    }
  };
#pragma unroll 1
  for (int st = 0; st < S; ++st)
    if (fetch_next() && tile >= 0) {
      valid |= 1u << st;
      if (lane == 0) {
        fetch(st, 0);
        if (C::APART) fetch(st, 1);
      }
    }

  // ---- per-lane offsets of the ldmatrix rows (see the swizzle: 16-byte piece c of row r sits at c ^ (r & 7),
  // or c ^ ((r >> 1) & 3) in 64-byte rows)
  constexpr bool NARROW = C::SWIZZLE_ROW == 64;
  auto row_off = [&](int row, int odd) -> uint32_t {  // row's start, with piece `odd` (0 or 1) swizzled
    const int x = NARROW ? (row >> 1) & 3 : row & 7;
    return row * C::SWIZZLE_ROW + ((odd ^ x) << 4);
  };
  // pieces 2 j and 2 j + 1 of the row: an even piece number is xored in, boxes hold 8 pieces of each row
  auto piece = [&](uint32_t base, uint32_t off, int j) -> uint32_t {
    return base + (NARROW ? 0 : (j >> 2) * C::BOX) + (off ^ ((NARROW ? 2 * j : (2 * j & 7)) << 4));
  };
  const uint32_t k_off = row_off((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4);
  // 8-bit values: bytes 4 t .. 4 t + 3 of a transposed row are to be tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9
  const uint32_t v_off = F8 ? row_off(2 * ((lane & 15) >> 2) + (lane & 1) + (lane & 2) * 4, lane >> 4)
                            : row_off((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1);

  uint32_t qf[C::QREG ? NT : 1][C::QREG ? KS : 1][2];
  uint2* q_sm = reinterpret_cast<uint2*>(sm + C::OFF_Q + wid * C::QBYTES);
  // m: reference of each of the lane's heads; qs: the score's factor.  8-bit pages: qh the part of that factor that
  // comes before the key's exponent, vr the values' reference (o is the sum times it), most what a score's place under
  // m and a value's exponent may come to together before vr is lowered
  float o[KS][NT][4], m[NT][2], l[NT][2], lost[NT][2], qs[NT][2], qh[NT][2], vr[NT][2], most[NT][2];
  const float log2e_scale = a.scale * 1.44269504088896340736f;
  int st = 0;

  // ================================================================ portions
#pragma unroll 1
  for (bool more = busy; more; more = out.next(a, w.p, sc)) {
    const int kvh = kv_head(w.p, out.hg), h0 = (out.hg - kvh * w.p.groups) * C::HEADS;
    const int nh = min(C::HEADS, a.n_rep - h0);
    const int64_t head0 = (int64_t)kvh * a.n_rep + h0;
    // ---- queries as B fragments: head g, dims 16 ks + 2 t, + 1 and + 8, + 9 (8-bit pages: 4 t .. 4 t + 3,
    // the order in which ldmatrix hands out the bytes of a key row)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + g;
      // heads that are none read the first one's row and become zero: loads without a branch go out together
      const uint16_t* qr = a.q + out.b * a.q_stride + (head0 + (h < nh ? h : 0)) * D;
      const uint32_t keep = h < nh ? 0xffffffffu : 0u;
      int e_up = 0;
      if (F8 && w.q_bf16) {
        uint32_t top = 0;
#pragma unroll 8
        for (int ks = 0; ks < KS; ++ks) {
          const uint2 x = *reinterpret_cast<const uint2*>(qr + ks * 16 + 4 * t);
          top = max(max(top, max(x.x & 0x7fffu, (x.x >> 16) & 0x7fffu)), max(x.y & 0x7fffu, (x.y >> 16) & 0x7fffu));
        }
        top = max(top, __shfl_xor_sync(kFull, top, 1));
        top = max(top, __shfl_xor_sync(kFull, top, 2));
        // largest entry in [2^14, 2^15); the factor is undone in the score's
        const int e = (int)(top >> 7) - 127;
        e_up = max(-126, min(14 - e, 126));
      }
      const float up = power2(e_up);
      // rolled where it can be: code that runs once costs its fetch, not its execution
#pragma unroll(C::QREG ? KS : 8)
      for (int ks = 0; ks < KS; ++ks) {
        uint2 x;
        if (F8) {
          x = *reinterpret_cast<const uint2*>(qr + ks * 16 + 4 * t);
        } else {
          x.x = *reinterpret_cast<const uint32_t*>(qr + ks * 16 + 2 * t);
          x.y = *reinterpret_cast<const uint32_t*>(qr + ks * 16 + 2 * t + 8);
        }
        if (F8 && w.q_bf16) {
          const __half2 u = __floats2half2_rn(__uint_as_float(x.x << 16) * up, __uint_as_float(x.x & 0xffff0000u) * up);
          const __half2 v = __floats2half2_rn(__uint_as_float(x.y << 16) * up, __uint_as_float(x.y & 0xffff0000u) * up);
          x = make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v));
        }
        x.x &= keep;
        x.y &= keep;
        if constexpr (C::QREG) {
          qf[nt][ks][0] = x.x;
          qf[nt][ks][1] = x.y;
        } else {
          q_sm[(nt * KS + ks) * 32 + lane] = x;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (F8) {
          const int e = __shfl_sync(kFull, e_up, (2 * t + i) * 4);
          qh[nt][i] = power2(-(e >> 1));
          qs[nt][i] = log2e_scale * power2((e >> 1) - e);
        } else {
          qs[nt][i] = log2e_scale;
        }
        m[nt][i] = kNone;
        vr[nt][i] = power2(kValueTop);
        most[nt][i] = kValueMost + kLazy - kValueTop;
        l[nt][i] = lost[nt][i] = 0.f;
      }
    }
    // pages of the segment that the sequence's end or the window cuts
    const int cut_first = out.s.lo % kPage ? 0 : -1, cut_last = out.s.len % kPage ? out.s.pages - 1 : -1;
    if constexpr (!C::QREG) __syncwarp();
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][nt][i] = 0.f;

    // ================================================================ pages
#pragma unroll 1
    for (int i = 0; i < out.take; ++i, st = st + 1 == S ? 0 : st + 1) {
      const bool here = valid >> st & 1;
      const uint32_t kb = stage0 + st * C::PAGE, vb = kb + (C::APART ? C::HALF : kPage * C::SWIZZLE_ROW);
      float s[NT][4];
      if (here) {  // with a limit of 0 the first copy is waited for
        const uint32_t limit = w.p.wait_limit || parity ? w.p.wait_limit : kDrainLimit;
        if ((parity & kLate) == 0 && !bar_wait(bar0 + 16 * st, parity >> st & 1, limit)) give_up(valid);
        parity ^= 1u << st;
      }
      int ek0 = 0, ek1 = 0, ev0 = 0, ev1 = 0;
      if (here) {
        if (F8) {  // exponents of tokens g and g + 8, keys and values
          const uint32_t ea = exp0 + st * C::EXP + g;
          asm volatile("ld.shared.s8 %0, [%1];" : "=r"(ek0) : "r"(ea) : "memory");
          asm volatile("ld.shared.s8 %0, [%1];" : "=r"(ek1) : "r"(ea + 8) : "memory");
          asm volatile("ld.shared.s8 %0, [%1];" : "=r"(ev0) : "r"(ea + 16) : "memory");
          asm volatile("ld.shared.s8 %0, [%1];" : "=r"(ev1) : "r"(ea + 24) : "memory");
        }
        float s2[NT][4];
        auto score = [&](int ks, const uint32_t(&af)[4], float(&acc)[NT][4]) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint2 x;
            if constexpr (C::QREG) x = make_uint2(qf[nt][ks][0], qf[nt][ks][1]);
            else x = q_sm[(nt * KS + ks) * 32 + lane];
            if (ks < 2) mma_first<BF>(acc[nt], af, x.x, x.y);
            else mma<BF>(acc[nt], af, x.x, x.y);
          }
        };
        if constexpr (F8) {
#pragma unroll
          for (int j = 0; j < KS / 2; ++j) {
            uint32_t r[4];
            ldsm4(r, piece(kb, k_off, j));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t af[4] = {f16_of_e4m3(r[2 * c]), f16_of_e4m3(r[2 * c + 1]), f16_of_e4m3_high(r[2 * c]),
                                      f16_of_e4m3_high(r[2 * c + 1])};
              if (c) score(2 * j + c, af, s2);
              else score(2 * j + c, af, s);
            }
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            uint32_t r[4];
            ldsm4(r, piece(kb, k_off, ks));
            if (ks & 1) score(ks, r, s2);
            else score(ks, r, s);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[nt][k] += s2[nt][k];
      }
      bool again = false;
      auto next_page = [&]() {
        __syncwarp();  // every lane has read what the copy replaces
        again = fetch_next() && tile >= 0;
        valid = again ? valid | 1u << st : valid & ~(1u << st);
        if (again && (parity & kLate) == 0 && lane == 0) fetch(st, 0);
      };
      if (C::APART) next_page();  // the keys are read

      if (here) {
        // ---- weights
        const int rel = out.p + i;  // page of the segment
        const bool whole = rel != cut_first && rel != cut_last;
        const int t_lo = out.s.lo - (out.s.first + rel) * kPage, t_hi = out.s.len - (out.s.first + rel) * kPage;
        auto counts = [&](int tok) { return tok >= t_lo && tok < t_hi; };
        if (F8) {
          const float f0 = power2(ek0), f1 = power2(ek1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[nt][k] = s[nt][k] * qh[nt][k & 1] * (k < 2 ? f0 : f1);
        }
        bool raise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[nt][k] *= qs[nt][k & 1];
        if (!whole) {  // rows that do not count are whatever memory held
          const bool ok0 = counts(g), ok1 = counts(g + 8);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[nt][k] = (k < 2 ? ok0 : ok1) ? s[nt][k] : -CUDART_INF_F;
          ev0 = ok0 ? ev0 : -127;
          ev1 = ok1 ? ev1 : -127;
        }
        const float fe0 = (float)ev0, fe1 = (float)ev1;
        float p[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            p[nt][k] = s[nt][k] - m[nt][k & 1];
            raise |= p[nt][k] > kLazy;
            if (F8) raise |= p[nt][k] + (k < 2 ? fe0 : fe1) > most[nt][k & 1];
          }
        if (__any_sync(kFull, raise)) {  // all heads' references are set anew: fewer pages come here
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float mx = fmaxf(s[nt][k], s[nt][k + 2]);
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, x));
              mx = fmaxf(m[nt][k], ceilf(mx));
              const float up = mx - m[nt][k], c = ex2(-up);
              m[nt][k] = mx;
              l[nt][k] *= c;
              if (C::KEEP_LOST) lost[nt][k] *= c;
              p[nt][k] = s[nt][k] - mx;
              p[nt][k + 2] = s[nt][k + 2] - mx;
              float co = c;
              if (F8) {  // the values' reference follows, and their sum takes what it does not
                float top = fmaxf(fmaxf(p[nt][k] + fe0, p[nt][k + 2] + fe1), -1000.f);
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, x));
                const int e = kValueMost + (int)kLazy - (int)most[nt][k], by = (int)fminf(up, 1000.f);
                const int e1 = max(min(min(e + by, kValueTop), kValueAt + (int)kLazy - (int)floorf(top)), kValueLeast);
                most[nt][k] = (float)(kValueMost + (int)kLazy - e1);
                vr[nt][k] = power2(e1);
                co = power2(max(e1 - e - by, -127));
              }
#pragma unroll
              for (int j = 0; j < KS; ++j) {
                o[j][nt][k] *= co;
                o[j][nt][k + 2] *= co;
              }
            }
        }
        // what a token's weight at its values has besides: 2^-8, and on 8-bit pages their exponent
        const float w0 = F8 ? power2(ev0) * kDown : kDown, w1 = F8 ? power2(ev1) * kDown : kDown;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int k = 0; k < 4; ++k) p[nt][k] = ex2(p[nt][k]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if constexpr (C::KEEP_LOST) {  // what an addition loses is kept for the next one (Kahan's sum)
              const float y = p[nt][k] + p[nt][k + 2] - lost[nt][k], sum = l[nt][k] + y;
              lost[nt][k] = sum - l[nt][k] - y;
              l[nt][k] = sum;
            } else {
              l[nt][k] += p[nt][k] + p[nt][k + 2];
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            p[nt][k] *= k < 2 ? w0 : w1;
            if (F8) p[nt][k] *= vr[nt][k & 1];
          }
        }
        constexpr int PARTS = BF ? 3 : 2;
        // 16-bit parts of tokens 0 .. 7 and 8 .. 15, or tf32 parts of tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9
        uint32_t pf[KIND == kF16 ? 1 : NT][PARTS][2], wh[KIND == kF16 ? NT : 1][4], wl[KIND == kF16 ? NT : 1][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (KIND == kF16) {
            turn(p[nt][0], p[nt][1]);
            turn(p[nt][2], p[nt][3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) tf32_parts(p[nt][k], wh[nt][k], wl[nt][k]);
          } else {
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
              pf[nt][k][0] = movmat(take_part<BF>(p[nt][0], p[nt][1]));
              pf[nt][k][1] = movmat(take_part<BF>(p[nt][2], p[nt][3]));
            }
          }
        }
        if (C::APART) {
          if ((parity & kLate) == 0 && !bar_wait(bar0 + 16 * st + 8, vparity >> st & 1, w.p.wait_limit)) give_up(valid | 1u << st);
          vparity ^= 1u << st;
        }
        if (!whole) {
          // value rows that do not count: a weight of 0 does not remove a NaN
#pragma unroll
          for (int k = 0; k < C::HALF / 512; ++k) {
            const uint32_t row = (k * 32 + lane) * 16 / C::SWIZZLE_ROW, col = (k * 32 + lane) * 16 % C::SWIZZLE_ROW;
            if (!counts(row % kPage))
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vb + row / kPage * C::BOX + row % kPage * C::SWIZZLE_ROW + col),
                           "r"(0)
                           : "memory");
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the stage's next copy
          __syncwarp();
        }
        auto add = [&](int j, const uint32_t(&af)[4]) {
          // af: dims g, g + 8 of tokens 2 t, 2 t + 1 (first two), 2 t + 8, 2 t + 9; a product of 8 tokens takes a
          // pair's first token as number t and its second as number t + 4
          uint32_t va[2][4];
          if constexpr (KIND == kF16)
#pragma unroll
            for (int k = 0; k < 4; ++k) widen(af[k], va[k >> 1][k & 1], va[k >> 1][(k & 1) + 2]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float acc[4];
            if constexpr (KIND != kF16) {
              mma_first<BF>(acc, af, pf[nt][PARTS - 1][0], pf[nt][PARTS - 1][1]);
#pragma unroll
              for (int k = PARTS - 2; k >= 0; --k) mma<BF>(acc, af, pf[nt][k][0], pf[nt][k][1]);
            } else {
              mma_tf32_first(acc, va[0], wl[nt][0], wl[nt][1]);
              mma_tf32(acc, va[1], wl[nt][2], wl[nt][3]);
              mma_tf32(acc, va[0], wh[nt][0], wh[nt][1]);
              mma_tf32(acc, va[1], wh[nt][2], wh[nt][3]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) o[j][nt][k] += acc[k];
          }
        };
        if constexpr (F8) {
#pragma unroll
          for (int j = 0; j < KS / 2; ++j) {
            uint32_t r[4];
            ldsm2t8(r, piece(vb, v_off, j));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t af[4] = {f16_of_e4m3(r[2 * c]), f16_of_e4m3(r[2 * c + 1]), f16_of_e4m3_high(r[2 * c]),
                                      f16_of_e4m3_high(r[2 * c + 1])};
              add(2 * j + c, af);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            uint32_t r[4];
            ldsm4t(r, piece(vb, v_off, j));
            add(j, r);
          }
        }
      }
      if (C::APART) {
        __syncwarp();
        if (again && (parity & kLate) == 0 && lane == 0) fetch(st, 1);
      } else {
        next_page();
      }
    }

    // ================================================================ the portion's result
    const bool dead = __any_sync(kFull, (parity & kLate) != 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][k] += __shfl_xor_sync(kFull, l[nt][k], x);
        if (dead) l[nt][k] = CUDART_NAN_F;
      }
    // The rows: to the outputs when the warp had the whole segment, else to its slot of shared memory.
    const bool begins = out.at == 0, all = begins && out.end == out.span;
    if (all && lane == 0) w.cuts[(int64_t)out.b * heads + out.hg] = make_int2(0, 0);
    const int64_t row = (int64_t)out.b * a.hq + head0;
    float* dst = all ? a.out + row * D : begins ? own_stage : own_slot;
    const int pitch = all ? D : C::PITCH;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int h = nt * 8 + 2 * t + k;
        if (h >= nh) continue;
        float* p = dst + h * pitch + g;  // accumulator rows g and g + 8 of tile j
        const float f = (all ? inverse_of(l[nt][k]) : 1.f) * (F8 ? power2(-exponent_in(vr[nt][k])) : 1.f);
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          p[16 * j] = o[j][nt][k] * f;
          p[16 * j + 8] = o[j][nt][k + 2] * f;
        }
        if (g == 0) {
          if (!all) ml[(begins * NW + wid) * C::HEADS + h] = make_float2(m[nt][k], l[nt][k]);
          else if (a.lse) a.lse[row + h] = lse_of(m[nt][k], l[nt][k]);
        }
      }
    // sequence, segment, whether it ends here, and where it ends on the line
    if (!all && lane == 0)
      rec[begins * NW + wid] = make_int4(out.b, out.hg, 1 + (out.end == out.span), x_end - out.left - out.at + out.span);
  }
  if (parity & kLate) flag_error(a.err, TQ_DEVERR_TIMEOUT);
  if (bad_id) flag_error(a.err, TQ_DEVERR_BLOCK_ID);

  // ================================================================ the CTA's cut segments
  // A run: the piece that begins a segment (or the first warp's, if it continues one) and the pieces of
  // the next warps that continue it.  A warp per (run, head).
  __syncthreads();
  const int4 r0 = lane < NW ? rec[lane] : make_int4(0, 0, 0, 0), r1 = lane < NW ? rec[NW + lane] : make_int4(0, 0, 0, 0);
  const uint32_t goes_on = __ballot_sync(kFull, r0.z != 0), stops = __ballot_sync(kFull, r0.z == 2);
  const uint32_t begun = __ballot_sync(kFull, r1.z != 0);
  const int runs = __popc(begun) + (goes_on & 1), per_run = min(C::HEADS, a.n_rep);
#pragma unroll 1
  for (int it = wid; it < runs * per_run; it += NW) {
    const int run = it / per_run, h = it - run * per_run;
    // the run's first warp, and whether it begins the segment
    const bool kind = !(run == 0 && (goes_on & 1));
    uint32_t left = begun;
    for (int k = goes_on & 1; k < run; ++k) left &= left - 1;
    const int lead = kind ? __ffs(left) - 1 : 0;
    const int seq = __shfl_sync(kFull, kind ? r1.x : r0.x, lead), hg = __shfl_sync(kFull, kind ? r1.y : r0.y, lead);
    const int ends_at = __shfl_sync(kFull, r1.w, lead);
    // the warps behind it that continue: as long as there are such, up to one that ends it
    const uint32_t on = lead < 31 ? goes_on >> (lead + 1) : 0, off = lead < 31 ? stops >> (lead + 1) : 0;
    int more = __ffs(~on) - 1;
    bool ends = !kind && (stops & 1);
    if (ends) more = 0;
    else if (off && __ffs(off) <= more) {
      more = __ffs(off);
      ends = true;
    }
    const int kvh = kv_head(w.p, hg), h0 = (hg - kvh * w.p.groups) * C::HEADS;
    if (h >= a.n_rep - h0) continue;
    // lane k: reference and total of warp k's piece
    const bool part_of = lane >= lead && lane <= lead + more;
    const float2 v = part_of ? ml[((lane == lead && kind) * NW + lane) * C::HEADS + h] : make_float2(-CUDART_INF_F, 0.f);
    float M, L = 0.f;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(M) : "f"(v.x));
    const float c = ex2(v.x - (M == -CUDART_INF_F ? 0.f : M)), cl = c * v.y;
    constexpr int V = D / 32, VL = V < 4 ? V : 4;
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = 0.f;
    const float* p = (kind ? reinterpret_cast<const float*>(sm + lead * S * C::PAGE)
                           : reinterpret_cast<const float*>(sm + C::OFF_SLOT)) + h * C::PITCH;
#pragma unroll 4
    for (int k = 0; k <= more; ++k) {
      const float f = __shfl_sync(kFull, c, lead + k);
      L += __shfl_sync(kFull, cl, lead + k);
#pragma unroll
      for (int i = 0; i < V; i += VL) {
        const float* q = p + (i / VL * 32 + lane) * VL;
        if constexpr (VL == 2) {
          const float2 y = *reinterpret_cast<const float2*>(q);
          x[0] = fmaf(f, y.x, x[0]);
          x[1] = fmaf(f, y.y, x[1]);
        } else {
          const float4 y = *reinterpret_cast<const float4*>(q);
          x[i] = fmaf(f, y.x, x[i]);
          x[i + 1] = fmaf(f, y.y, x[i + 1]);
          x[i + 2] = fmaf(f, y.z, x[i + 2]);
          x[i + 3] = fmaf(f, y.w, x[i + 3]);
        }
      }
      p = reinterpret_cast<const float*>(sm + C::OFF_SLOT) + ((lead + k + 1) * C::HEADS + h) * C::PITCH;
    }
    // a whole segment goes to the outputs; else the CTA's slot of its kind: [HEADS][D] sums, then references
    // and totals
    const bool all = kind && ends;
    const int64_t row = (int64_t)seq * a.hq + (int64_t)kvh * a.n_rep + h0 + h;
    float* part = w.parts + ((int64_t)blockIdx.x * 2 + kind) * (C::HEADS * (D + 2));
    float* dst = all ? a.out + row * D : part + h * D;
    const float f = all ? inverse_of(L) : 1.f;
#pragma unroll
    for (int i = 0; i < V; i += VL) {
      float* q = dst + (i / VL * 32 + lane) * VL;
      if constexpr (VL == 2) *reinterpret_cast<float2*>(q) = make_float2(x[0] * f, x[1] * f);
      else *reinterpret_cast<float4*>(q) = make_float4(x[i] * f, x[i + 1] * f, x[i + 2] * f, x[i + 3] * f);
    }
    if (lane == 0) {
      if (!all) {
        part[C::HEADS * D + h] = M;
        part[C::HEADS * (D + 1) + h] = L;
      } else if (a.lse) {
        a.lse[row] = lse_of(M, L);
      }
      // the last CTA with a piece of it: the one with the last cut more than tau before its end
      if (kind && h == 0)
        w.cuts[(int64_t)seq * heads + hg] = make_int2(blockIdx.x, ends ? blockIdx.x : (pieces.from(ends_at - kTau) - 1) / NW);
    }
  }
}

// Joins the pieces of the segments that more than one team had, and writes the rows of empty sequences.
// JOIN warps share a (segment, query head): with few segments of many pieces all of a CTA's, a CTA per head; with
// many of few pieces one warp for all heads of a segment.  A lane has D / 32 dims, four pieces are loaded
// at a time: what bounds this kernel is the chain of loads from L2, segment -> pieces, and nothing else.
constexpr int kMergeWarps = 4;
template <int D, int HEADS, int JOIN>
__global__ void __launch_bounds__((JOIN == 1 ? kMergeWarps : JOIN) * 32) paged_merge_kernel(const __grid_constant__ PagedWork w, int segments) {
  constexpr int V = D / 32, VL = V < 4 ? V : 4;  // dims of a lane, and of one load
  constexpr int PART = HEADS * (D + 2);
  const PagedArgs& a = w.a;
  __shared__ __align__(16) float sx[JOIN == 1 ? 1 : JOIN][D];
  __shared__ float sl[JOIN], sm_max[JOIN];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const unsigned seg = JOIN == 1 ? blockIdx.x * kMergeWarps + wid : blockIdx.x;
  if (seg >= (unsigned)segments) return;
  const unsigned heads = a.hkv * w.p.groups;
  const int2 cut = w.cuts[seg];
  const int b = seg / heads, hg = seg - b * heads;
  const int pages = seq_of(a, a.lengths[b]).pages;
  const int kvh = kv_head(w.p, hg), h0 = (hg - kvh * w.p.groups) * HEADS, nh = min(HEADS, a.n_rep - h0);
  const int64_t row0 = (int64_t)b * a.hq + (int64_t)kvh * a.n_rep + h0;
  const int n = pages ? cut.y - cut.x + 1 : 0;  // CTAs that had pieces of it
  if (n == 1) return;
  // the first CTA's second slot, the first slots of those behind
  const float* part0 = w.parts + (int64_t)cut.x * 2 * PART;
  for (int h = JOIN == 1 ? 0 : blockIdx.y; h < nh; h += JOIN == 1 ? 1 : gridDim.y) {
    float M = -CUDART_INF_F, L = 0.f, x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = 0.f;
    for (int k0 = JOIN == 1 ? 0 : wid; k0 < n; k0 += 4 * JOIN) {
      float m[4], l[4], y[4][V];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = k0 + u * JOIN;
        m[u] = -CUDART_INF_F;
        l[u] = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) y[u][i] = 0.f;
        if (k >= n) continue;
        const float* p = part0 + (k == 0 ? 1 : 2 * k) * (int64_t)PART;
        m[u] = p[HEADS * D + h];
        l[u] = p[HEADS * (D + 1) + h];
#pragma unroll
        for (int i = 0; i < V; i += VL) {
          const float* q = p + h * D + (i / VL * 32 + lane) * VL;
          if constexpr (VL == 2) {
            const float2 v = *reinterpret_cast<const float2*>(q);
            y[u][0] = v.x;
            y[u][1] = v.y;
          } else {
            const float4 v = *reinterpret_cast<const float4*>(q);
            y[u][i] = v.x;
            y[u][i + 1] = v.y;
            y[u][i + 2] = v.z;
            y[u][i + 3] = v.w;
          }
        }
      }
      const float top = fmaxf(fmaxf(M, fmaxf(m[0], m[1])), fmaxf(m[2], m[3]));
      const float sub = top == -CUDART_INF_F ? 0.f : top, c = ex2(M - sub);
      M = top;
      L *= c;
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] *= c;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float f = ex2(m[u] - sub);
        L = fmaf(f, l[u], L);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = fmaf(f, y[u][i], x[i]);
      }
    }
    if constexpr (JOIN > 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) sx[wid][(i / VL * 32 + lane) * VL + i % VL] = x[i];
      if (lane == 0) {
        sl[wid] = L;
        sm_max[wid] = M;
      }
      __syncthreads();
      M = sm_max[0];
#pragma unroll
      for (int k = 1; k < JOIN; ++k) M = fmaxf(M, sm_max[k]);
      const float sub = M == -CUDART_INF_F ? 0.f : M;
      float c[JOIN];
      L = 0.f;
#pragma unroll
      for (int k = 0; k < JOIN; ++k) {
        c[k] = ex2(sm_max[k] - sub);
        L = fmaf(c[k], sl[k], L);
      }
      const float f = inverse_of(L);
      for (int i = threadIdx.x; i < D; i += JOIN * 32) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < JOIN; ++k) v = fmaf(c[k], sx[k][i], v);
        a.out[(row0 + h) * D + i] = v * f;
      }
      if (threadIdx.x == 0 && a.lse) a.lse[row0 + h] = lse_of(M, L);
      if (h + (int)gridDim.y < nh) __syncthreads();
    } else {
      const float f = inverse_of(L);
#pragma unroll
      for (int i = 0; i < V; ++i) a.out[(row0 + h) * D + (i / VL * 32 + lane) * VL + i % VL] = x[i] * f;
      if (lane == 0 && a.lse) a.lse[row0 + h] = lse_of(M, L);
    }
  }
}

// ---------------------------------------------------------------- host side
template <int KIND, int D, int NT>
PagedPlan plan_of(const tq_ctx* ctx) {
  using C = PagedCfg<KIND, D, NT>;
  PagedPlan p;
  const int n_rep = ctx->cfg.num_q_heads / ctx->cfg.num_kv_heads;
  p.groups = (n_rep + C::HEADS - 1) / C::HEADS;
  p.teams = ctx->sm_count * C::NW;
  p.unit = 0;
  p.wait_limit = ctx->wait_limit;
  return p;
}

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// The CTAs' slots, then the segments' cuts.
template <int KIND, int D, int NT>
size_t parts_bytes(const PagedPlan& p) {
  using C = PagedCfg<KIND, D, NT>;
  return align256((size_t)(p.teams / C::NW) * 2 * C::HEADS * (D + 2) * 4);
}
template <int KIND, int D, int NT>
size_t workspace_of(const tq_ctx* ctx, int batch) {
  const PagedPlan p = plan_of<KIND, D, NT>(ctx);
  return parts_bytes<KIND, D, NT>(p) + align256((size_t)batch * ctx->cfg.num_kv_heads * p.groups * sizeof(int2));
}

template <int KIND, int D, int NT>
cudaError_t launch_one(tq_ctx* ctx, const PagedArgs& a, void* workspace, cudaStream_t s) {
  using C = PagedCfg<KIND, D, NT>;
  PagedWork w;
  w.a = a;
  w.p = plan_of<KIND, D, NT>(ctx);
  w.q_bf16 = ctx->cfg.key_format == TQ_ELEM_BF16;
  w.parts = static_cast<float*>(workspace);
  w.cuts = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + parts_bytes<KIND, D, NT>(w.p));  // for all CTAs
  // The longest line these arguments allow: the unit keeps it below 2^31, and a short one gets no more CTAs than
  // it has use for.
  const int64_t all = (int64_t)a.batch * a.hkv * w.p.groups;
  int64_t pages = a.max_blocks;
  if (a.window && pages > ((int64_t)a.window + 2 * kPage - 2) / kPage) pages = ((int64_t)a.window + 2 * kPage - 2) / kPage;
  while (all * ((pages >> w.p.unit) + 1 + kLead) > 0x7fffffff)
    if (++w.p.unit > 27) return cudaErrorInvalidValue;
  const int64_t line = all * ((pages >> w.p.unit) + 1 + kLead), want = (line + C::NW - 1) / C::NW;
  const int ctas = want < ctx->sm_count ? (int)want : ctx->sm_count;
  w.p.teams = ctas * C::NW;
  CUtensorMap map{};
  if (a.num_blocks > 0) {
    const PagedTensorMap tm{a.pool, C::ES, D, (int64_t)a.num_blocks * a.hkv, C::PAGE + C::EXP, C::SWIZZLE_ROW, C::BOX_ROWS};
    if (!encode_paged_map(tm, &map)) return cudaErrorInvalidValue;
  }
  auto kern = paged_kernel<KIND, D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  prof_start(ctx, kProfDecode, s);
  e = launch_early(kern, dim3(ctas), dim3(C::THREADS), C::SMEM, s, map, w);
  prof_stop(ctx, kProfDecode, s);
  if (e != cudaSuccess) return e;
  ctx->launches++;
  ctx->decode_kernel = "paged_kernel";

  const int segments = a.batch * a.hkv * w.p.groups;
  const bool many = segments >= 4 * ctx->sm_count;
  const dim3 each(segments, a.n_rep < C::HEADS ? a.n_rep : C::HEADS);  // a CTA per (segment, head)
  prof_start(ctx, kProfMerge, s);
  if (many)
    e = launch_early(paged_merge_kernel<D, C::HEADS, 1>, dim3((segments + kMergeWarps - 1) / kMergeWarps), dim3(kMergeWarps * 32), 0, s, w,
                     segments);
  else if (24 * segments > ctx->sm_count)
    e = launch_early(paged_merge_kernel<D, C::HEADS, kMergeWarps>, each, dim3(kMergeWarps * 32), 0, s, w, segments);
  else  // up to all CTAs' pieces in one segment (2 segments of 2900 pages, 76 pieces each: 5 us with 4 warps)
    e = launch_early(paged_merge_kernel<D, C::HEADS, 16>, each, dim3(16 * 32), 0, s, w, segments);
  prof_stop(ctx, kProfMerge, s);
  if (e == cudaSuccess) ctx->launches++;
  return e;
}

// Query heads per segment: 8, or 16 when a KV head has more than 8 (d = 512: always 8, for want of registers).
template <int KIND>
cudaError_t launch_kind(tq_ctx* ctx, const PagedArgs& a, void* ws, cudaStream_t s) {
  const bool two = a.n_rep > 8;
  switch (ctx->cfg.head_dim) {
    case 64: return two ? launch_one<KIND, 64, 2>(ctx, a, ws, s) : launch_one<KIND, 64, 1>(ctx, a, ws, s);
    case 128: return two ? launch_one<KIND, 128, 2>(ctx, a, ws, s) : launch_one<KIND, 128, 1>(ctx, a, ws, s);
    case 256: return two ? launch_one<KIND, 256, 2>(ctx, a, ws, s) : launch_one<KIND, 256, 1>(ctx, a, ws, s);
    case 512: return launch_one<KIND, 512, 1>(ctx, a, ws, s);
  }
  return cudaErrorInvalidValue;
}

template <int KIND>
size_t workspace_kind(const tq_ctx* ctx, int batch) {
  const bool two = ctx->cfg.num_q_heads / ctx->cfg.num_kv_heads > 8;
  switch (ctx->cfg.head_dim) {
    case 64: return two ? workspace_of<KIND, 64, 2>(ctx, batch) : workspace_of<KIND, 64, 1>(ctx, batch);
    case 128: return two ? workspace_of<KIND, 128, 2>(ctx, batch) : workspace_of<KIND, 128, 1>(ctx, batch);
    case 256: return two ? workspace_of<KIND, 256, 2>(ctx, batch) : workspace_of<KIND, 256, 1>(ctx, batch);
    case 512: return workspace_of<KIND, 512, 1>(ctx, batch);
  }
  return 0;
}

}  // namespace
}  // namespace tq
