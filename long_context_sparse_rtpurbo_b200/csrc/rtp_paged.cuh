// Decode step of one layer over a paged cache: the G query heads of a KV head attend to the
// rows of a sequence's pages, every position for retrieval heads, the sinks and the window for
// local heads:
//   z_n = R(m) q . k_n / sqrt(128),  o = sum_n softmax(z)_n v_n,  lse = log sum_n exp(z_n).
//
// Bound by HBM: 512 B (bf16) or 264 B (e4m3 rows and their scales) per attended row against
// 4 * 128 * G flops. So the rows are read once for the G heads, through per-warp rings of
// asynchronous copies, and the arithmetic on them stays in one warp's registers.
//
// Work split: a group is a (sequence, KV head) pair, a tile 16 rows. The tiles of all groups
// form one line, cut into equal ranges for the CTAs and again for their warps, whatever the
// lengths are. A warp runs its range as one pipeline across group borders; groups that lie
// inside its range are written straight out. What remains open at a warp's two ends is merged
// in shared memory, and what remains open at a CTA's two ends goes to the workspace, where the
// CTA that arrives last at a group merges its parts in the order of the line (no waits, and the
// result does not depend on who is last).
//
// Measured (8 KV heads of 4 query heads, all dense; launches back to back): 1M tokens in bf16
// 627 us, 6.85 TB/s (without the arithmetic 609 us); 4 x 128K tokens in e4m3 187 us, 5.9 TB/s
// (173 us). Under a load of seconds the power limit takes the clock from 1965 to about 1700 MHz:
// 638 to 656 us, and e4m3, which follows the clock, 202 to 217 us. One sequence of 4K tokens takes 11 us: the chain of lengths, page
// ids, rows, two joins and an arrival, each a trip to L2 or memory.
#pragma once

#include "rtp_attend.cuh"
#include "rtp_append.cuh"

namespace rtp {

constexpr int kKvBf16 = 0, kKvE4m3 = 1;
constexpr int kPagedMaxCTAs = 160;
constexpr int kPagedMaxRanges = 2 * kPagedMaxCTAs;
constexpr int kLaterShare = 8;              // 1 / this of a long line is left to the CTAs done first
constexpr int kPagedCtrlBytes = 4096;       // status word at 0, arrival counters from 256
constexpr int kPagedReserveCounter = 960;   // word index of the reservation's arrival counter
constexpr int kPagedQueue = 961;            // word index of the decode step's queue of later ranges
constexpr float kE4m3Max = 448.f;
constexpr float kScaleMin = 1.17549435e-38f;   // 2^-126

struct PagedPtrs {
  unsigned char *k, *v;          // [n_pages] pages of [Hkv][page][128], page_stride rows apart
  float *ks, *vs;                // e4m3: [n_pages][Hkv][page]
  const int32_t* table;          // [B][table_stride]
  int page_stride;               // rows; all rows are below 2^31
  int table_stride, n_pages, lg; // page = 1 << lg
};

struct PagedDecodeParams {
  LayerShape L;
  PagedPtrs C;
  const uint16_t *q_pre, *k_new, *v_new;
  const int32_t* seq_lens;
  uint16_t* out;
  float* lse;
  int* status;
  uint32_t *arrive, *queue;
  float *part, *head;            // [ranges][2] partials of ranges, [CTAs][16] of warps
};

// bf16 rows: 8 warps with three tiles each, 192 KB of copies in the rings; the query's terms alone
// are 48 registers a thread. (12 warps with two tiles each: 3 % slower on short sequences.)
// e4m3 rows: their conversions keep the SM busy, so more warps: 12 with four tiles each, 187 us at
// 4 x 131072 tokens of 8 KV heads; 8 warps 248 us, 16 warps (128 registers, some spilled) 191 us.
template <int KV> struct PagedCfg;
template <> struct PagedCfg<kKvBf16> {
  static constexpr int kWarps = 8, kStages = 3, kRowB = 256, kTerms = 3;
  static constexpr int kStageB = 16 * 512;
  static constexpr int kLift = 0;
  static constexpr bool kLater = true;         // ranges for the CTAs done first
};
template <> struct PagedCfg<kKvE4m3> {
  static constexpr int kWarps = 12, kStages = 4, kRowB = 128, kTerms = 2;
  static constexpr int kStageB = 16 * 256 + 128;
  // The accumulators' weights are lifted by 2^6: fp16 terms end at 2^-24, so that a row below 2^-25
  // of the reference would not count in the output (128K such rows under one that weighs 2^26 as
  // much: 2 % of the output). Lifted, a weight is off by 2^-31 of the reference at most; their
  // bound of 2^9 becomes 2^15, within fp16.
  static constexpr int kLift = 6;
  static constexpr bool kLater = false;
};

constexpr int kPagedMaxWarps = 16;
// Tiles' worth of a group's fixed cost (query, angles, output) in the split of the line: 256
// sequences of 0 to 1024 tokens took 145 us without it, 115 us with 3 (and with 8)
constexpr int kSetup = 3;
static_assert(kSetup > 0, "an empty sequence is divided by its places");

// floats of a warp's partial (rows of 132: the accumulators' lanes hit all banks) and of a CTA's
constexpr int kPartPitch = 132;
__host__ __device__ constexpr int warp_part_floats(int G) { return G * kPartPitch + 32; }
__host__ __device__ constexpr int cta_part_floats(int G) { return G * kD + 32; }
__host__ __device__ constexpr size_t paged_part_floats(int G) {
  return (size_t)2 * kPagedMaxRanges * cta_part_floats(G) +
         (size_t)kPagedMaxCTAs * kPagedMaxWarps * warp_part_floats(G);
}

struct PagedEntry {              // an open end of a warp's range
  long long gs, ge;              // its group on the line: first tile, end
  int gid;                       // sequence * Hkv + position of the KV head in the group order; -1: none
  int pad;
};

// Places a warp from which on a share of the line is left to the CTAs done first
constexpr int kLaterPlaces = 128;
// Tiles per warp up to which a group stays in one CTA, where every group can have one
constexpr int kOneCta = 5;

template <int KV>
struct PagedSmem {
  using Cfg = PagedCfg<KV>;
  static constexpr int kEntries = 2 * Cfg::kWarps;
  static_assert(kEntries <= 32, "a warp's lanes stand for the entries");
  static constexpr int kRing = Cfg::kWarps * Cfg::kStages * Cfg::kStageB;
  static constexpr int kTheta = kRing;                             // [64] doubles
  static constexpr int kAng = kTheta + 64 * 8;                     // [warps][64] (cos, sin)
  static constexpr int kMask = kAng + Cfg::kWarps * 64 * 8;        // [warps][8] row masks
  static constexpr int kEnt = kMask + Cfg::kWarps * 8 * 4;
  static constexpr int kPrefix = kEnt + kEntries * (int)sizeof(PagedEntry);   // [129]
  static constexpr int kMisc = kPrefix + 130 * 8;
  static constexpr int kWt = kMisc + 256;                          // [ranges][8] weights of a merge
  static constexpr int kBytes = kWt + (Cfg::kLater ? kPagedMaxRanges : kPagedMaxCTAs) * 8 * 4;
  static_assert(2 * warp_part_floats(8) * 4 <= Cfg::kStages * Cfg::kStageB, "a drained ring holds two partials");
};

// Lets the stream's next launch be set up while this one runs, and waits for the launches before
// this one: nothing is read or written before that. (Launches one after another otherwise start
// about 2 us apart at the least; a decode step's append then takes 4.1 us instead of 6.2.)
__device__ __forceinline__ void launch_begin() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A parameter's element by its generic address, all lanes at once: loads from the constant bank
// take one address at a time (an append of 32K e4m3 tokens: 69 us with those, 56 us with these)
__device__ __forceinline__ double ld_gen(const double* p) {
  double x;
  asm("ld.f64 %0, [%1];" : "=d"(x) : "l"(p));
  return x;
}
__device__ __forceinline__ double2 ld_gen(const double2* p) {
  double2 x;
  asm("ld.v2.f64 {%0, %1}, [%2];" : "=d"(x.x), "=d"(x.y) : "l"(p));
  return x;
}
// z turned on by w: the product of two (cos, sin)
__device__ __forceinline__ double2 turned(double2 z, double2 w) {
  return make_double2(z.x * w.x - z.y * w.y, z.y * w.x + z.x * w.y);
}

// ------------------------------------------------------------------ conversions and products

__device__ __forceinline__ uint32_t pack_h2(float x, float y) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
// (x, y) = hi + lo in fp16
__device__ __forceinline__ void split_h2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_h2(x, y);
  const __half2 h = *reinterpret_cast<const __half2*>(&hi);
  lo = pack_h2(x - __low2float(h), y - __high2float(h));
}
// two e4m3 bytes -> fp16x2, exact
__device__ __forceinline__ uint32_t e4m3x2_h2(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t;}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_h2_hi(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %1; cvt.rn.f16x2.e4m3x2 %0, b;}" : "=r"(r) : "r"(w));
  return r;
}
// float -> e4m3, nearest even, values beyond +-448 to +-448
__device__ __forceinline__ uint32_t f_e4m3x2(float x, float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16-byte copy that writes zeros where n = 0 (the address is not read then)
__device__ __forceinline__ void cp_async16_zf(uint32_t saddr, const void* gmem, uint32_t n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(saddr), "l"(gmem), "r"(n)
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 2^(a - b), 0 where a is the empty state's -inf
__device__ __forceinline__ float ex2_from(float a, float b) { return a == -INFINITY ? 0.f : ex2(a - b); }
__device__ __forceinline__ uint32_t low_mask(int n) { return (1u << min(max(n, 0), 16)) - 1u; }

// The stored scale of a row: amax / 448 in single precision, at least 2^-126 (a zero row).
// The quotient by a rounded reciprocal and Markstein's correction by the exact remainder: rounded
// once (448 q is a multiple of 2^-143, so the remainder is exact; compared with the division for
// every float).
__device__ __forceinline__ float row_scale(float amax) {
  constexpr float inv = 1.f / kE4m3Max;
  const float q = amax * inv, r = fmaf(-kE4m3Max, q, amax);
  return fmaxf(amax < INFINITY ? fmaf(r, inv, q) : amax, kScaleMin);
}

// Eight values as e4m3 bytes of x / scale, inv = 1 / scale rounded. The quotient in single
// precision, rounded once: an estimate and Markstein's correction by its exact remainder, two
// values an instruction. Where the remainder could be too small a number for that, the values are
// divided.
__device__ __forceinline__ uint2 e4m3_of8(const float* x, float scale, float inv) {
  float q[8];
  unsigned long long s2, i2;
  asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(-scale));
  asm("mov.b64 %0, {%1, %1};" : "=l"(i2) : "f"(inv));
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    unsigned long long x2, q2, r2;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x2) : "f"(x[e]), "f"(x[e + 1]));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q2) : "l"(x2), "l"(i2));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r2) : "l"(q2), "l"(s2), "l"(x2));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q2) : "l"(r2), "l"(i2), "l"(q2));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(q[e]), "=f"(q[e + 1]) : "l"(q2));
  }
  if (scale < 1e-25f || !(scale < 1e38f)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = __fdiv_rn(x[e], scale);
  }
  return make_uint2(f_e4m3x2(q[0], q[1]) | f_e4m3x2(q[2], q[3]) << 16,
                    f_e4m3x2(q[4], q[5]) | f_e4m3x2(q[6], q[7]) << 16);
}

// ------------------------------------------------------------------ the line of tiles

// Length of sequence b; 0 (no tiles) for an empty or an invalid one.
__device__ __forceinline__ int paged_len(const PagedDecodeParams& P, int b, bool* bad) {
  if (b >= P.L.B) return 0;
  const int n = P.seq_lens[b];
  const int64_t cap = min((int64_t)P.C.table_stride << P.C.lg, P.L.maxN);
  if (n < 0 || n > cap) { if (bad) *bad = true; return 0; }
  return n;
}

// Tiles of a local head: those of the sinks, then those of the window that come after them.
struct LocalTiles { int ns, sh, lo, nt; };
__device__ __forceinline__ LocalTiles local_tiles(const LayerShape& L, int n) {
  LocalTiles t;
  const int tr = (n + 15) >> 4;
  t.ns = min((int)(((int64_t)L.sinks + 15) >> 4), tr);
  t.lo = max(0, n - L.window);
  const int wt = max(t.ns, t.lo >> 4);
  t.sh = wt - t.ns;
  t.nt = t.ns + tr - wt;
  return t;
}
// Length of a sequence on the line: a group is kSetup places without a tile, then its tiles.
__device__ __forceinline__ long long seq_places(const LayerShape& L, int n) {
  if (n <= 0) return 0;
  return (long long)L.n_ret * (((n + 15) >> 4) + kSetup) +
         (long long)L.n_loc * (local_tiles(L, n).nt + kSetup);
}

// A place on the line. Sequences are in batch order; in a sequence the retrieval KV heads come
// first. lens: this lane's length of the 32 sequences around b.
struct Cursor {
  int b, gi, k, nt, n, lens;
  int ns, sh, lo;                // tile k covers rows from 16 (k < ns ? k : k + sh); window from lo
  int kvrow;                     // first row of the KV head in a page
  const int32_t* pages;          // the sequence's page ids
};

__device__ __forceinline__ int kv_head(const LayerShape& L, int gi) {
  return gi < L.n_ret ? L.ret_kv[gi] : L.loc_kv[gi - L.n_ret];
}
__device__ __forceinline__ void cursor_group(const PagedDecodeParams& P, Cursor& c) {
  const LayerShape& L = P.L;
  c.kvrow = kv_head(L, min(c.gi, L.Hkv - 1)) << P.C.lg;
  c.pages = P.C.table + (int64_t)c.b * P.C.table_stride;
  if (c.gi < L.n_ret) {
    c.ns = 0; c.sh = 0; c.lo = 0; c.nt = (c.n + 15) >> 4;
  } else {
    const LocalTiles t = local_tiles(L, c.n);
    c.ns = t.ns; c.sh = t.sh; c.lo = t.lo; c.nt = t.nt;
  }
}
__device__ __forceinline__ void cursor_next_group(const PagedDecodeParams& P, Cursor& c) {
  c.k = 0;
  if (++c.gi == P.L.Hkv) {
    c.gi = 0;
    do {
      ++c.b;
      if ((c.b & 31) == 0) c.lens = paged_len(P, c.b + (threadIdx.x & 31), nullptr);
      c.n = __shfl_sync(0xffffffffu, c.lens, c.b & 31);
    } while (c.n == 0 && c.b < P.L.B);
  }
  cursor_group(P, c);
}
// a / b for a quotient below 2^20: an estimate, off by one at most, and its correction
__device__ __forceinline__ int small_div(int a, int b) {
  int q = (int)(__fdividef((float)a, (float)b));
  const int r = a - q * b;
  return q + (r >= b) - (r < 0);
}

// The cursor of the first tile at or after a place of the line, rel places after the start of a
// chunk of 32 sequences (not at its end). lens: this lane's length of the chunk; incl and mine: its
// places with and without the lanes before. *skip: places from there to the tile.
__device__ __forceinline__ Cursor cursor_at(const PagedDecodeParams& P, int chunk, long long rel,
                                            int lens, long long incl, long long mine, int* skip) {
  Cursor c;
  c.lens = lens;
  const int j = __popc(__ballot_sync(0xffffffffu, incl <= rel)) & 31;
  c.b = chunk * 32 + j;
  c.n = __shfl_sync(0xffffffffu, lens, j);
  const int in_seq = (int)(rel - __shfl_sync(0xffffffffu, incl - mine, j));
  const int tr = ((c.n + 15) >> 4) + kSetup;
  int k;
  if (in_seq < P.L.n_ret * tr) {
    c.gi = small_div(in_seq, tr);
    k = in_seq - c.gi * tr;
  } else {
    const int u = in_seq - P.L.n_ret * tr, tl = local_tiles(P.L, c.n).nt + kSetup;
    c.gi = small_div(u, tl);
    k = u - c.gi * tl;
    c.gi += P.L.n_ret;
  }
  *skip = max(kSetup - k, 0);
  c.k = max(k - kSetup, 0);
  cursor_group(P, c);
  return c;
}
// The next tile, and its place
__device__ __forceinline__ void cursor_step(const PagedDecodeParams& P, Cursor& c, int& place) {
  ++place;
  if (++c.k == c.nt) {
    cursor_next_group(P, c);
    place += kSetup;
  }
}
template <class I>
__device__ __forceinline__ I warp_incl_sum(I x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I u = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += u;
  }
  return x;
}

// The line cut into ranges: n equal ones, one for each CTA (the first `extra` of them a place
// longer), and behind place T1 n2 smaller ones, which the CTAs that are done first take.
// Plain 64-bit divisions cost about 500 cycles each here; one is left, for lines beyond 2^32.
struct LineSplit {
  long long each, T1;
  int n, extra, n2, each2, extra2;
};
template <bool LATER>
__device__ __forceinline__ LineSplit split_line(long long T, int n, int n2) {
  if (!LATER) n2 = 0;
  LineSplit s;
  s.n = n;
  s.n2 = n2;
  s.T1 = n2 ? T - T / kLaterShare : T;
  s.each = s.T1 >> 32 ? s.T1 / n : (long long)((uint32_t)s.T1 / (uint32_t)n);
  s.extra = (int)(s.T1 - s.each * n);
  s.each2 = n2 ? (int)((T - s.T1) / n2) : 0;
  s.extra2 = n2 ? (int)(T - s.T1 - (long long)s.each2 * n2) : 0;
  return s;
}
template <bool LATER>
__device__ __forceinline__ long long range_start(const LineSplit& s, int i) {
  if (!LATER || i < s.n) return s.each * i + min(i, s.extra);
  i -= s.n;
  return s.T1 + (long long)s.each2 * i + min(i, s.extra2);
}
// The range that holds a place: a quotient is at most 160, so its single-precision estimate is
// off by one at most.
template <bool LATER>
__device__ __forceinline__ int range_of(const LineSplit& s, long long place) {
  const bool later = LATER && place >= s.T1;
  const long long x = later ? place - s.T1 : place, each = later ? s.each2 : s.each;
  const int extra = later ? s.extra2 : s.extra, n = later ? s.n2 : s.n;
  int i = min((int)__fdividef((float)x, (float)(each + 1)), n - 1);
  if (i >= extra) i = min(extra + (int)__fdividef((float)(x - extra * (each + 1)), (float)each), n - 1);
  if (each * i + min(i, extra) > x) --i;
  if (i + 1 < n && each * (i + 1) + min(i + 1, extra) <= x) ++i;
  return later ? s.n + i : i;
}

struct TileDesc { int pid, row; uint32_t mask; };   // page, row in the page block, rows attended
__device__ __forceinline__ TileDesc tile_desc(const PagedDecodeParams& P, const Cursor& c) {
  const int pos = 16 * (c.k < c.ns ? c.k : c.k + c.sh);
  TileDesc d;
  d.pid = c.pages[pos >> P.C.lg];
  d.row = c.kvrow + (pos & ((1 << P.C.lg) - 1));
  d.mask = 0xffffu;
  if (pos + 16 > c.n || pos < c.lo)                    // the end, the window's edges
    d.mask = low_mask(c.n - pos) & (low_mask(P.L.sinks - pos) | ~low_mask(c.lo - pos));
  return d;
}

// Starts the copies of a tile into a stage of this warp's ring; *mask_slot gets its row mask.
// Rows that are not attended become zeros, so that what a page holds there (NaN included) takes
// no part. Each copy instruction moves 512 contiguous bytes; 16-byte chunks are XOR-swizzled by
// the row, so that the ldmatrix reads of eight rows hit all banks.
template <int KV>
__device__ __forceinline__ void tile_issue(const PagedDecodeParams& P, const TileDesc& d,
                                           uint32_t stage, uint32_t* mask_slot) {
  using Cfg = PagedCfg<KV>;
  const int lane = threadIdx.x & 31;
  uint32_t mask = d.mask;
  int pid = d.pid;
  if ((uint32_t)pid >= (uint32_t)P.C.n_pages) {        // a page that does not exist: no rows
    if (lane == 0) set_status(P.status, -6);
    mask = 0;
    pid = 0;
  }
  if (lane == 0) *mask_slot = mask;
  const int64_t off = (int64_t)(pid * P.C.page_stride + d.row) * Cfg::kRowB + lane * 16;
  const unsigned char* kp = P.C.k + off;
  const unsigned char* vp = P.C.v + off;
  constexpr int kCh = Cfg::kRowB / 16;                 // chunks per row: 16 or 8
  const int r0 = lane / kCh, c0 = lane % kCh;          // rows of one instruction: 2 or 4
  constexpr int kRows = 32 / kCh;
  const uint32_t dst = stage + r0 * Cfg::kRowB;
  const uint32_t sw = (uint32_t)(c0 ^ r0) << 4;
  if (mask == 0xffffu) {
#pragma unroll
    for (int u = 0; u < 16 / kRows; ++u) {
      const uint32_t s = dst + u * 512 + (sw ^ (uint32_t)(((u * kRows) & 7) << 4));
      cp_async16_s(s, kp + u * 512);
      cp_async16_s(s + 16 * Cfg::kRowB, vp + u * 512);
    }
  } else {
#pragma unroll
    for (int u = 0; u < 16 / kRows; ++u) {
      const uint32_t s = dst + u * 512 + (sw ^ (uint32_t)(((u * kRows) & 7) << 4));
      const uint32_t n = (mask >> (u * kRows + r0)) & 1u ? 16u : 0u;
      cp_async16_zf(s, kp + u * 512, n);
      cp_async16_zf(s + 16 * Cfg::kRowB, vp + u * 512, n);
    }
  }
  if (KV == kKvE4m3 && lane < 8) {                     // 16 scales of K, then of V
    const float* sp = (lane < 4 ? P.C.ks : P.C.vs) + (pid * (P.L.Hkv << P.C.lg) + d.row + (lane & 3) * 4);
    cp_async16_s(stage + 32 * Cfg::kRowB + lane * 16, sp);
  }
}

// ------------------------------------------------------------------ one warp's attention

// Softmax state of a group's heads 2t and 2t + 1 (t = lane % 4) and the O^T accumulators. The
// weights of the sum l are 2^(z - m). Those of the accumulators are 2^(z + log2(v scale) - mo),
// with mo = m in a bf16 cache: the references are separate because rows carry their own scale, and
// mo is kLift below the maximum that it stands for.
template <int KV>
struct PagedAttn {
  float acc[8][4];
  float m[2], l[2], mo[2];
  uint32_t q[8][2 * PagedCfg<KV>::kTerms];     // B fragments of Q^T, one pair per term
  float qf[2];                                 // e4m3: power of two taken out of the heads' query
  float cf[2];                                 // e4m3: 2^(m - mo)
};

template <int KV>
__device__ __forceinline__ void attn_reset(PagedAttn<KV>& A) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) A.acc[i][e] = 0.f;
#pragma unroll
  for (int e = 0; e < 2; ++e) { A.m[e] = A.mo[e] = -INFINITY; A.l[e] = 0.f; A.cf[e] = INFINITY; }
}

// (cos, sin) of the query position's 64 angles into this warp's table. theta lies in shared
// memory: lanes that read different words of the parameters would be served one by one.
__device__ __forceinline__ void fill_angles(const double* theta, float2* ang, int pos) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float s, c;
    rope_sincosf((double)pos, theta[lane + 32 * e], &s, &c);
    ang[lane + 32 * e] = make_float2(c, s);
  }
  __syncwarp();
}

// This lane's channels of the head's query: pairs c..c+1 (and 64 on) of the first and second
// half of each 16-channel step of the products.
template <int KV>
__device__ __forceinline__ int query_channel(int kk, int e) {
  const int t = threadIdx.x & 3;
  return KV == kKvBf16 ? 16 * kk + 2 * t + 8 * e : 16 * kk + 4 * t + 2 * e;
}
struct QueryRaw { uint32_t lo[8], hi[8]; };
template <int KV>
__device__ __forceinline__ void query_fetch(const PagedDecodeParams& P, QueryRaw& R, int b, int g) {
  const int h = (threadIdx.x & 31) >> 2, G = P.L.G;
  const uint16_t* q = P.q_pre + ((int64_t)b * P.L.Hq + (int64_t)g * G + min(h, G - 1)) * kD;
#pragma unroll
  for (int kk = 0; kk < 4; ++kk)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = query_channel<KV>(kk, e);
      R.lo[2 * kk + e] = *reinterpret_cast<const uint32_t*>(q + i);
      R.hi[2 * kk + e] = *reinterpret_cast<const uint32_t*>(q + i + 64);
    }
}

// R(m) q log2(e) / sqrt(128) of the G heads as B fragments. bf16 cache: three bf16 terms (24
// bits). e4m3 cache: two fp16 terms (22 bits) of the query divided by a power of two that
// brings its largest element into [1, 2), since fp16 has few exponents.
template <int KV>
__device__ __forceinline__ void query_terms(PagedAttn<KV>& A, const QueryRaw& R, const float2* ang,
                                            int G) {
  const int lane = threadIdx.x & 31, h = lane >> 2, t = lane & 3;
  const float sc = kLog2e * 0.08838834764831845f;      // 1 / sqrt(128)
  float x[8][4];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t lo = R.lo[2 * kk + e], hi = R.hi[2 * kk + e];
      const float4 a = *reinterpret_cast<const float4*>(ang + query_channel<KV>(kk, e));
      x[kk][2 * e] = (bf_lo(lo) * a.x - bf_lo(hi) * a.y) * sc;
      x[kk][2 * e + 1] = (bf_hi(lo) * a.z - bf_hi(hi) * a.w) * sc;
      x[kk + 4][2 * e] = (bf_lo(lo) * a.y + bf_lo(hi) * a.x) * sc;
      x[kk + 4][2 * e + 1] = (bf_hi(lo) * a.w + bf_hi(hi) * a.z) * sc;
    }
  if (h >= G) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[kk][e] = 0.f;
  }
  if (KV == kKvE4m3) {
    float mx = 0.f;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
      for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(x[kk][e]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int ex = min(max((int)(__float_as_uint(mx) >> 23), 1), 253);
    const float down = __uint_as_float((uint32_t)(254 - ex) << 23);
    const float up = __uint_as_float((uint32_t)ex << 23);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        split_h2(x[kk][2 * e] * down, x[kk][2 * e + 1] * down, A.q[kk][e], A.q[kk][2 + e]);
    A.qf[0] = __shfl_sync(0xffffffffu, up, 8 * t);
    A.qf[1] = __shfl_sync(0xffffffffu, up, 8 * t + 4);
  } else {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float a = x[kk][2 * e], b2 = x[kk][2 * e + 1];
        const uint32_t hi = pack_bf2(a, b2);
        const float ra = a - bf_lo(hi), rb = b2 - bf_hi(hi);
        A.q[kk][e] = hi;
        split_bf2(ra, rb, A.q[kk][2 + e], A.q[kk][(KV == kKvBf16 ? 4 : 0) + e]);
      }
  }
}

// Moves a reference: x holds this lane's logits of the two heads (rows g, g + 8). It only moves
// when a logit is more than 2^8 above it (the weights then stay below 2^8), so most tiles cost
// one vote instead of the maximum over the rows. LIFT: how far the reference lies below the maximum.
template <int LIFT>
__device__ __forceinline__ bool move_ref(const float (&x)[4], float (&m)[2], float (&al)[2]) {
  const float t0 = m[0] + (8.f + LIFT), t1 = m[1] + (8.f + LIFT);
  const bool up = x[0] > t0 || x[2] > t0 || x[1] > t1 || x[3] > t1;
  if (!__any_sync(0xffffffffu, up)) return false;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float mx = fmaxf(x[e], x[2 + e]);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m[e], mx - LIFT);
    al[e] = mn == -INFINITY ? 1.f : ex2(m[e] - mn);
    m[e] = mn;
  }
  return true;
}

// One tile of 16 rows. Logits S^T = K Q^T, weights as B operand of O^T += V^T P^T in two terms: a
// weight is off by 2^-17 (two bf16 terms) or 2^-22 (two fp16 terms, and see kLift) of itself, where
// the output is rounded by up to 2^-8; a third term would be half as many products again. The sum l
// and the accumulators are in single precision.
template <int KV>
__device__ __forceinline__ void paged_tile(PagedAttn<KV>& A, uint32_t stage, uint32_t mask) {
  using Cfg = PagedCfg<KV>;
  const int lane = threadIdx.x & 31, g = lane >> 2;
  const uint32_t tv = stage + 16 * Cfg::kRowB;
  float x[4];
  float vs[2] = {0.f, 0.f};
  if (KV == kKvBf16) {
    float s[3][4];
#pragma unroll
    for (int j = 0; j < 3; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
    const int r = lane & 15;
    const uint32_t ka = stage + r * 256 + (uint32_t)(((lane >> 4) ^ (r & 7)) << 4);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      uint32_t a[4];
      ldsm_x4(ka ^ (uint32_t)(kk << 5), a);
#pragma unroll
      for (int j = 0; j < 3; ++j) mma_bf16(s[j], a, A.q[kk][2 * j], A.q[kk][2 * j + 1]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = s[0][e] + (s[1][e] + s[2][e]);
  } else {
    float s[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
    const int r = lane & 15;
    const uint32_t ka = stage + r * 128 + (uint32_t)(((lane >> 4) ^ (r & 7)) << 4);
    uint32_t wk[4][4];                                 // (all loads first: 6 % on the whole step)
#pragma unroll
    for (int i = 0; i < 4; ++i) ldsm_x4(ka ^ (uint32_t)(i << 5), wk[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t (&w)[4] = wk[i];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t a[4] = {e4m3x2_h2(w[2 * c]), e4m3x2_h2(w[2 * c + 1]),
                               e4m3x2_h2_hi(w[2 * c]), e4m3x2_h2_hi(w[2 * c + 1])};
#pragma unroll
        for (int j = 0; j < 2; ++j)
          mma_f16(s[j], a, A.q[2 * i + c][2 * j], A.q[2 * i + c][2 * j + 1]);
      }
    }
    const uint32_t sc = stage + 32 * Cfg::kRowB + g * 4;
    float k0, k1;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(k0) : "r"(sc) : "memory");
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(k1) : "r"(sc + 32) : "memory");
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vs[0]) : "r"(sc + 64) : "memory");
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vs[1]) : "r"(sc + 96) : "memory");
    x[0] = (s[0][0] + s[1][0]) * (k0 * A.qf[0]);
    x[1] = (s[0][1] + s[1][1]) * (k0 * A.qf[1]);
    x[2] = (s[0][2] + s[1][2]) * (k1 * A.qf[0]);
    x[3] = (s[0][3] + s[1][3]) * (k1 * A.qf[1]);
  }
  if (mask != 0xffffu) {
    if (!((mask >> g) & 1u)) { x[0] = x[1] = -INFINITY; vs[0] = 0.f; }
    if (!((mask >> (g + 8)) & 1u)) { x[2] = x[3] = -INFINITY; vs[1] = 0.f; }
  }
  float al[2] = {1.f, 1.f};
  const bool moved = move_ref<0>(x, A.m, al);
  float p[4];
  {
    const float m0 = A.m[0] == -INFINITY ? 0.f : A.m[0], m1 = A.m[1] == -INFINITY ? 0.f : A.m[1];
    p[0] = ex2(x[0] - m0); p[1] = ex2(x[1] - m1);
    p[2] = ex2(x[2] - m0); p[3] = ex2(x[3] - m1);
  }
  if (moved) { A.l[0] *= al[0]; A.l[1] *= al[1]; }
  A.l[0] += p[0] + p[2];
  A.l[1] += p[1] + p[3];
  bool moved_o = moved;
  if (KV == kKvE4m3) {
    // The rows' weights with their scales, against their own reference: 2^(x + log2(vs) - mo) =
    // p vs 2^(m - mo). A weight above 2^(9 + kLift) moves the reference; so does a factor above 2^64,
    // whose p could have been too small a number.
    if (moved) { A.cf[0] = ex2(A.m[0] - A.mo[0]); A.cf[1] = ex2(A.m[1] - A.mo[1]); }
    const float f0 = vs[0] * A.cf[0], f1 = vs[0] * A.cf[1], f2 = vs[1] * A.cf[0], f3 = vs[1] * A.cf[1];
    const float w0 = p[0] * f0, w1 = p[1] * f1, w2 = p[2] * f2, w3 = p[3] * f3;
    const bool far = !((f0 + f1) + (f2 + f3) <= 1.8446744e19f) ||
                     !((w0 + w1) + (w2 + w3) <= (float)(512 << Cfg::kLift));
    moved_o = __any_sync(0xffffffffu, far);
    if (moved_o) {
      const float lv0 = lg2(vs[0]), lv1 = lg2(vs[1]);  // -inf for rows that are left out
      const float y[4] = {x[0] + lv0, x[1] + lv0, x[2] + lv1, x[3] + lv1};
      al[0] = al[1] = 1.f;
      move_ref<Cfg::kLift>(y, A.mo, al);
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = ex2_from(y[e], A.mo[e & 1]);
      A.cf[0] = ex2(A.m[0] - A.mo[0]);
      A.cf[1] = ex2(A.m[1] - A.mo[1]);
    } else {
      p[0] = w0; p[1] = w1; p[2] = w2; p[3] = w3;
    }
  } else {
    A.mo[0] = A.m[0];
    A.mo[1] = A.m[1];
  }
  if (moved_o) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      A.acc[i][0] *= al[0]; A.acc[i][1] *= al[1];
      A.acc[i][2] *= al[0]; A.acc[i][3] *= al[1];
    }
  }
  uint32_t h01, l01, h23, l23;
  if (KV == kKvBf16) {
    split_bf2(p[0], p[1], h01, l01);
    split_bf2(p[2], p[3], h23, l23);
  } else {
    split_h2(p[0], p[1], h01, l01);
    split_h2(p[2], p[3], h23, l23);
  }
  const uint32_t bh0 = movm_t(h01), bh1 = movm_t(h23);
  const uint32_t bl0 = movm_t(l01), bl1 = movm_t(l23);
  if (KV == kKvBf16) {
    const int j = lane >> 3, r = (lane & 7) + (j >> 1) * 8;
    const uint32_t va = tv + r * 256 + (uint32_t)(((j & 1) ^ (lane & 7)) << 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t a[4];
      ldsm_x4_t(va ^ (uint32_t)(i << 5), a);
      mma_bf16(A.acc[i], a, bh0, bh1);
      mma_bf16(A.acc[i], a, bl0, bl1);
    }
  } else {
    // a transposed 16-bit element is a pair of channels (2 g, 2 g + 1) of one token: row g of
    // the product takes the even channel, row g + 8 the odd one
    const int r = lane & 15;
    const uint32_t va = tv + r * 128 + (uint32_t)(((lane >> 4) ^ (r & 7)) << 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[4];
      ldsm_x4_t(va ^ (uint32_t)(i << 5), w);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t u0 = __byte_perm(w[2 * c], 0, 0x3120), u1 = __byte_perm(w[2 * c + 1], 0, 0x3120);
        const uint32_t a[4] = {e4m3x2_h2(u0), e4m3x2_h2_hi(u0), e4m3x2_h2(u1), e4m3x2_h2_hi(u1)};
        mma_f16(A.acc[2 * i + c], a, bh0, bh1);
        mma_f16(A.acc[2 * i + c], a, bl0, bl1);
      }
    }
  }
}

// Channel of accumulator element e (0..3) of 16-channel block i in this lane
template <int KV>
__device__ __forceinline__ int acc_channel(int i, int e) {
  const int g = (threadIdx.x & 31) >> 2;
  return KV == kKvBf16 ? 16 * i + g + 8 * (e >> 1) : 16 * i + 2 * g + (e >> 1);
}

// What turns a sum of accumulators into the output: 2^(mo - m) / l, 0 where no row was attended. (The
// lift is taken out by itself: 2^(mo - m) is flushed to 0 below 2^-126.)
template <int KV>
__device__ __forceinline__ float out_factor(float m, float mo, float l) {
  constexpr int kLift = PagedCfg<KV>::kLift;
  return l > 0.f || l != l ? ex2_from(mo + kLift, m) / l * (1.f / (1 << kLift)) : 0.f;
}

// The sum over the rows of each head (a lane has those of rows g and g + 8 of every tile)
template <int KV>
__device__ __forceinline__ void attn_sum(PagedAttn<KV>& A) {
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) A.l[e] += __shfl_xor_sync(0xffffffffu, A.l[e], o);
}

// Output rows of a group that this warp holds whole
template <int KV>
__device__ __forceinline__ void attn_write(const PagedDecodeParams& P, const PagedAttn<KV>& A,
                                           int b, int g) {
  const int lane = threadIdx.x & 31, t = lane & 3, gr = lane >> 2, G = P.L.G;
  const int64_t head0 = (int64_t)b * P.L.Hq + (int64_t)g * G;
  float f[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) f[e] = out_factor<KV>(A.m[e], A.mo[e], A.l[e]);
  if (P.lse && gr == 0) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (2 * t + e < G) P.lse[head0 + 2 * t + e] = (A.m[e] + log2f(A.l[e])) * 0.6931471805599453f;
  }
  if (KV == kKvBf16) {
    // transposed in registers: a lane then has two neighbouring channels of head gr
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t w = movm_t(pack_bf2(A.acc[i][2 * u] * f[0], A.acc[i][2 * u + 1] * f[1]));
        if (gr < G)
          *reinterpret_cast<uint32_t*>(P.out + (head0 + gr) * kD + 16 * i + 8 * u + 2 * t) = w;
      }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (2 * t + e < G)
          *reinterpret_cast<uint32_t*>(P.out + (head0 + 2 * t + e) * kD + 16 * i + 2 * gr) =
              pack_bf2(A.acc[i][e] * f[e], A.acc[i][2 + e] * f[e]);
  }
}

// A partial in shared memory: [G][132] accumulators, then (m, l, mo) per head
template <int KV>
__device__ __forceinline__ void attn_store(const PagedAttn<KV>& A, float* dst, int G) {
  const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int h = 2 * t + e;
    if (h < G) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dst[h * kPartPitch + acc_channel<KV>(i, e)] = A.acc[i][e];
        dst[h * kPartPitch + acc_channel<KV>(i, 2 + e)] = A.acc[i][2 + e];
      }
      if ((lane >> 2) == 0) {
        float* ml = dst + G * kPartPitch + 3 * h;
        ml[0] = A.m[e]; ml[1] = A.l[e]; ml[2] = A.mo[e];
      }
    }
  }
}

// ------------------------------------------------------------------ the new token's row

// Writes the decode token's key and value of KV head g at its page row and into its row of the
// staged tile (one warp). The rotation and the roundings are those of the bulk append.
template <int KV>
__device__ __noinline__ void paged_append_row(const PagedDecodeParams& P, const double* theta, int b,
                                              int g, int pos, int64_t row, int64_t srow,
                                              uint32_t stage) {
  using Cfg = PagedCfg<KV>;
  const int lane = threadIdx.x & 31, r = pos & 15;
  const uint16_t* kp = P.k_new + ((int64_t)b * P.L.Hkv + g) * kD;
  const uint16_t* vp = P.v_new + ((int64_t)b * P.L.Hkv + g) * kD;
  const uint32_t kt = stage + r * Cfg::kRowB, vt = kt + 16 * Cfg::kRowB;
  unsigned char* kd = P.C.k + row * Cfg::kRowB;
  unsigned char* vd = P.C.v + row * Cfg::kRowB;
  // lane: channels 2 lane, 2 lane + 1 and their partners 64 on
  const uint32_t a = *reinterpret_cast<const uint32_t*>(kp + 2 * lane);
  const uint32_t c = *reinterpret_cast<const uint32_t*>(kp + 64 + 2 * lane);
  const uint32_t va = *reinterpret_cast<const uint32_t*>(vp + 2 * lane);
  const uint32_t vc = *reinterpret_cast<const uint32_t*>(vp + 64 + 2 * lane);
  double lo[2], hi[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    double sn, cs;
    rope_sincos((double)pos, theta[2 * lane + e], &sn, &cs);
    const double xa = e ? bf_hi(a) : bf_lo(a), xb = e ? bf_hi(c) : bf_lo(c);
    lo[e] = xa * cs - xb * sn;
    hi[e] = xa * sn + xb * cs;
  }
  const uint32_t sw = (uint32_t)(r & 7) << 4;
  if (KV == kKvBf16) {
    const uint32_t kl = d2bf_rn(lo[0]) | (uint32_t)d2bf_rn(lo[1]) << 16;
    const uint32_t kh = d2bf_rn(hi[0]) | (uint32_t)d2bf_rn(hi[1]) << 16;
    *reinterpret_cast<uint32_t*>(kd + 4 * lane) = kl;
    *reinterpret_cast<uint32_t*>(kd + 128 + 4 * lane) = kh;
    *reinterpret_cast<uint32_t*>(vd + 4 * lane) = va;
    *reinterpret_cast<uint32_t*>(vd + 128 + 4 * lane) = vc;
    const uint32_t o = (4u * lane) ^ sw;
    st_shared_u32(kt + o, kl);
    st_shared_u32(kt + (o ^ 128u), kh);
    st_shared_u32(vt + o, va);
    st_shared_u32(vt + (o ^ 128u), vc);
  } else {
    float x[2][4] = {{(float)lo[0], (float)lo[1], (float)hi[0], (float)hi[1]},
                     {bf_lo(va), bf_hi(va), bf_lo(vc), bf_hi(vc)}};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float mx = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(x[j][e]));
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float sc = row_scale(mx);
      const uint32_t w0 = f_e4m3x2(__fdiv_rn(x[j][0], sc), __fdiv_rn(x[j][1], sc));
      const uint32_t w1 = f_e4m3x2(__fdiv_rn(x[j][2], sc), __fdiv_rn(x[j][3], sc));
      unsigned char* d = j ? vd : kd;
      *reinterpret_cast<uint16_t*>(d + 2 * lane) = (uint16_t)w0;
      *reinterpret_cast<uint16_t*>(d + 64 + 2 * lane) = (uint16_t)w1;
      const uint32_t o = (2u * lane) ^ sw;
      const uint32_t tb = j ? vt : kt;
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(tb + o), "h"((uint16_t)w0) : "memory");
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(tb + (o ^ 64u)), "h"((uint16_t)w1) : "memory");
      if (lane == 0) {
        (j ? P.C.vs : P.C.ks)[srow] = sc;
        st_shared_u32(stage + 32 * Cfg::kRowB + 64 * j + 4 * r, __float_as_uint(sc));
      }
    }
  }
  __syncwarp();
}

// ------------------------------------------------------------------ the kernel

// Outputs of the sequences of a chunk that have no tiles (each by one CTA), and the report of
// lengths out of range. One warp.
__device__ __noinline__ void paged_idle(const PagedDecodeParams& P, int ch, int len, bool bad) {
  const int lane = threadIdx.x & 31, b = ch * 32 + lane;
  if (bad && blockIdx.x == 0) set_status(P.status, -6);
  uint32_t none = __ballot_sync(0xffffffffu, b < P.L.B && len == 0 && b % gridDim.x == blockIdx.x);
  while (none) {
    const int64_t e = ch * 32 + __ffs(none) - 1;
    none &= none - 1;
    uint4* o = reinterpret_cast<uint4*>(P.out + e * P.L.Hq * kD);
    for (int i = lane; i < P.L.Hq * (kD / 8); i += 32) o[i] = make_uint4(0, 0, 0, 0);
    if (P.lse)
      for (int i = lane; i < P.L.Hq; i += 32) P.lse[e * P.L.Hq + i] = -INFINITY;
  }
}

template <int KV, bool APPEND>
__global__ void __launch_bounds__(PagedCfg<KV>::kWarps * 32, 1)
paged_decode_kernel(const __grid_constant__ PagedDecodeParams P) {
  using Cfg = PagedCfg<KV>;
  using S = PagedSmem<KV>;
  constexpr int NW = Cfg::kWarps, NT = NW * 32, NS = Cfg::kStages;
  extern __shared__ __align__(1024) unsigned char sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const LayerShape& L = P.L;
  const int G = L.G;
  long long* prefix = reinterpret_cast<long long*>(sm + S::kPrefix);
  PagedEntry* ent = reinterpret_cast<PagedEntry*>(sm + S::kEnt);
  double* theta = reinterpret_cast<double*>(sm + S::kTheta);
  float2* ang = reinterpret_cast<float2*>(sm + S::kAng) + warp * 64;
  uint32_t* masks = reinterpret_cast<uint32_t*>(sm + S::kMask) + warp * 8;

  // ---- the line: places before each 32 sequences, and in all. Up to 32 sequences: every warp
  // makes the sums itself.
  const int nc = (L.B + 31) >> 5;
  int lens = 0, chunk = 0;
  long long mine = 0, incl = 0, base = 0, T;
  launch_begin();
  if (tid < 2 * NW) ent[tid].gid = -1;
  bool bad = false;
  if (nc == 1) lens = paged_len(P, lane, &bad);
  // while the lengths are on their way (the short way, 0.3 us less of 11, made the registers of the
  // e4m3 kernel come out 3 % slower on long lines)
  if (KV == kKvBf16) {
    if (tid < kD / 2) theta[tid] = ld_gen(&L.theta[tid]);
  } else if (lane == 0) {
#pragma unroll
    for (int i = 0; i < (kD / 2 + NW - 1) / NW; ++i)
      if (warp + i * NW < kD / 2) theta[warp + i * NW] = L.theta[warp + i * NW];
  }
  if (nc == 1) {
    const uint32_t m = (uint32_t)seq_places(L, lens), in = warp_incl_sum(m);   // below 2^32
    mine = m;
    incl = in;
    T = __shfl_sync(0xffffffffu, in, 31);
    if (warp == 0) paged_idle(P, 0, lens, bad);
  } else {
    for (int ch = warp; ch < nc; ch += NW) {
      bad = false;
      const int n = paged_len(P, ch * 32 + lane, &bad);
      const long long t = warp_incl_sum(seq_places(L, n));
      if (lane == 31) prefix[ch] = t;
      paged_idle(P, ch, n, bad);
    }
    __syncthreads();
    if (warp == 0) {                                   // exclusive sums, the total at [nc]
      long long run = 0;
      for (int c0 = 0; c0 < nc; c0 += 32) {
        const long long m = c0 + lane < nc ? prefix[c0 + lane] : 0;
        const long long in = warp_incl_sum(m);
        if (c0 + lane < nc) prefix[c0 + lane] = run + in - m;
        run += __shfl_sync(0xffffffffu, in, 31);
      }
      if (lane == 0) prefix[nc] = run;
    }
    __syncthreads();
    T = prefix[nc];
  }
  if (T == 0) return;
  // ---- this CTA's range
  long long ct0, ct1;
  LineSplit split;
  int* next_range = reinterpret_cast<int*>(sm + S::kMisc + 112);
  int range = blockIdx.x, later = 0;                   // later: ranges that are left to whoever is first
  {
    const uint32_t live = __ballot_sync(0xffffffffu, lens > 0);
    const int x = nc > 1 ? 0 : __reduce_max_sync(0xffffffffu, L.n_ret ? (lens + 15) >> 4 : local_tiles(L, lens).nt);
    if (nc == 1 && x <= kOneCta * NW && __popc(live) * L.Hkv <= gridDim.x) {
      // Few short groups: one CTA each. Joining the parts of several CTAs takes 4 us, as much as
      // 5 tiles of a warp.
      if (blockIdx.x >= __popc(live) * L.Hkv) return;
      const int s = small_div(blockIdx.x, L.Hkv), gi = blockIdx.x - s * L.Hkv;
      const int j = __ffs(__ballot_sync(0xffffffffu, lens > 0 && __popc(live & ((1u << lane) - 1)) == s)) - 1;
      const int n = __shfl_sync(0xffffffffu, lens, j), tr = ((n + 15) >> 4) + kSetup;
      const int tl = local_tiles(L, n).nt + kSetup;
      ct0 = __shfl_sync(0xffffffffu, incl - mine, j) + min(gi, L.n_ret) * tr + max(gi - L.n_ret, 0) * tl;
      ct1 = ct0 + (gi < L.n_ret ? tr : tl);
      // (no split: no group is left open); the places without a tile would leave warps idle
      ct0 += kSetup;
    } else {
      // All CTAs, as far as each warp gets a place. With few sequences a group's parts are what
      // counts in the end: spread over c CTAs, a group of x tiles takes a warp x / (c NW) tiles of
      // 0.8 us, and the CTA that joins it c parts of 13 ns a head; best at c^2 = 64 x / (NW G).
      int ctas = gridDim.x;
      if (T < (long long)ctas * NW) ctas = ((int)T + NW - 1) / NW;
      if (nc == 1 && T < (1 << 20))
        ctas = min(ctas, (int)(sqrtf(64.f / (NW * G) / (float)x) * (float)T) + 1);
      // The SMs get unequal shares of the bandwidth (15 % more and less than the median). On a long
      // line the CTAs that are done first take what was left for that, range by range: 4 % with
      // bf16 rows. (Not with e4m3 rows, whose SMs are busy computing and more even; and a line
      // of 57 places a warp lost 6 % to the joins of the additional ranges.)
      if (Cfg::kLater && ctas == gridDim.x && T >= (long long)ctas * NW * kLaterPlaces) later = ctas;
      split = split_line<Cfg::kLater>(T, ctas, later);
      if (blockIdx.x >= split.n) return;
      ct0 = range_start<Cfg::kLater>(split, blockIdx.x);
      ct1 = range_start<Cfg::kLater>(split, blockIdx.x + 1);
    }
  }
  unsigned char* ring = sm + warp * NS * Cfg::kStageB;
  const uint32_t ring_s = smem_u32(ring);
  auto entry_part = [&](int j) {
    return reinterpret_cast<const float*>(sm + (j >> 1) * NS * Cfg::kStageB) + (j & 1) * warp_part_floats(G);
  };

#pragma unroll 1
  while (true) {
    const int len = (int)(ct1 - ct0);                    // below 2^31: a sequence has 2^26 places at most
    // this warp's places, counted from ct0
    int line = (int)((long long)warp * len / NW);        // place of the tile at cc
    const int p1 = (int)((long long)(warp + 1) * len / NW);
    Cursor cc;
    if (line < p1) {
      const long long p0 = ct0 + line;
      if (nc > 1) {
        int before = 0;                                  // chunks that start at or before p0
        for (int i = lane; i < nc; i += 32) before += prefix[i] <= p0;
        chunk = __reduce_add_sync(0xffffffffu, before) - 1;
        base = prefix[chunk];
      }
      if (nc > 1 || (Cfg::kLater && range != blockIdx.x)) {
        lens = paged_len(P, chunk * 32 + lane, nullptr);
        mine = seq_places(L, lens);
        incl = warp_incl_sum(mine);
      }
      int skip;
      cc = cursor_at(P, chunk, p0 - base, lens, incl, mine, &skip);
      line += skip;
    }
    __syncthreads();                                     // theta, ent

    PagedAttn<KV> A;
    if (line < p1) {
      Cursor pc = cc;
      int pline = line;                                  // place of the tile at pc, the next to copy
      // fill the ring: the page ids of its tiles are loaded together, and the first query and its
      // angles meanwhile
      TileDesc d[NS];
      bool have[NS];
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        have[s] = pline < p1;
        if (have[s]) {
          d[s] = tile_desc(P, pc);
          cursor_step(P, pc, pline);
        }
      }
      QueryRaw qr;
      query_fetch<KV>(P, qr, cc.b, kv_head(L, cc.gi));
      fill_angles(theta, ang, cc.n - 1);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        if (have[s]) tile_issue<KV>(P, d[s], ring_s + s * Cfg::kStageB, masks + s);
        cp_async_commit();
      }
      TileDesc nx;                                       // the next tile, its page id on the way
      bool more = pline < p1;
      if (more) {
        nx = tile_desc(P, pc);
        cursor_step(P, pc, pline);
      }
      query_terms<KV>(A, qr, ang, G);
      attn_reset<KV>(A);
      int seg_k = cc.k, ang_b = cc.b, slot = 0;
      bool has_head = false, fresh = false;
#pragma unroll 1
      while (line < p1) {
        const int kvh = kv_head(L, cc.gi);
        if (fresh) {                                     // first tile of a group
          QueryRaw q2;
          query_fetch<KV>(P, q2, cc.b, kvh);
          if (cc.b != ang_b) {
            fill_angles(theta, ang, cc.n - 1);
            ang_b = cc.b;
          }
          query_terms<KV>(A, q2, ang, G);
          attn_reset<KV>(A);
          seg_k = 0;
          fresh = false;
        }
        cp_async_wait<NS - 1>();
        __syncwarp();
        const uint32_t stage = ring_s + slot * Cfg::kStageB;
        const uint32_t mask = masks[slot];
        if (APPEND && cc.k == cc.nt - 1 && mask) {       // the last tile holds the new token's row
          const int pos = cc.n - 1;
          const int pid = P.C.table[(int64_t)cc.b * P.C.table_stride + (pos >> P.C.lg)];
          const int in = (kvh << P.C.lg) + (pos & ((1 << P.C.lg) - 1));
          paged_append_row<KV>(P, theta, cc.b, kvh, pos, pid * P.C.page_stride + in,
                               pid * (L.Hkv << P.C.lg) + in, stage);
        }
        paged_tile<KV>(A, stage, mask);
        __syncwarp();
        if (more) {
          tile_issue<KV>(P, nx, stage, masks + slot);
          more = pline < p1;
          if (more) {
            nx = tile_desc(P, pc);
            cursor_step(P, pc, pline);
          }
        }
        cp_async_commit();
        if (++slot == NS) slot = 0;
        ++cc.k;
        ++line;
        const bool ends = cc.k == cc.nt;
        const bool last = line + (ends ? kSetup : 0) >= p1;
        if (ends || last) {
          attn_sum<KV>(A);
          const bool starts = seg_k == 0;
          if (starts && ends) {
            attn_write<KV>(P, A, cc.b, kvh);
          } else {
            // an open end: to the drained ring, or, where tiles of other groups follow and the ring
            // is in use, to the workspace for now (then it is of a group that an earlier warp began)
            float* dst = reinterpret_cast<float*>(ring) + (starts ? warp_part_floats(G) : 0);
            if (!last) {
              dst = P.head + (int64_t)(blockIdx.x * NW + warp) * warp_part_floats(G);
              has_head = true;
            } else {
              cp_async_wait<0>();
              __syncwarp();
            }
            attn_store<KV>(A, dst, G);
            if (lane == 0) {
              PagedEntry e;
              e.gid = cc.b * L.Hkv + cc.gi;
              e.ge = ct0 + line + (cc.nt - cc.k);
              e.gs = e.ge - cc.nt;
              e.pad = 0;
              ent[2 * warp + (starts ? 1 : 0)] = e;
            }
          }
          if (ends) {
            line += kSetup;
            if (!last) cursor_next_group(P, cc);
            fresh = true;
          }
        }
      }
      cp_async_wait<0>();
      __syncwarp();
      if (has_head) {
        const float4* src = reinterpret_cast<const float4*>(
            P.head + (int64_t)(blockIdx.x * NW + warp) * warp_part_floats(G));
#pragma unroll 9
        for (int i = lane; i < warp_part_floats(G) / 4; i += 32)
          reinterpret_cast<float4*>(ring)[i] = src[i];
      }
    }
    __syncthreads();

    // ---- the open ends of this CTA's warps: the entries of a group (a run) are merged in the order
    // of the line, one (run, head) a warp. (The code is kept small: it runs once, and most of its
    // time is that of fetching its instructions.)
    int open_run[2] = {-1, -1};                          // first entry of the groups left open
    {
      const int gid = lane < 2 * NW ? ent[lane].gid : -1;
      const uint32_t valid = __ballot_sync(0xffffffffu, gid >= 0), below = valid & ((1u << lane) - 1);
      const int before = __shfl_sync(0xffffffffu, gid, below ? 31 - __clz(below) : 0);
      const bool lead = gid >= 0 && (!below || before != gid);
      const uint32_t leads = __ballot_sync(0xffffffffu, lead);
      const PagedEntry* mine_e = ent + min(lane, 2 * NW - 1);
      const uint32_t left = __ballot_sync(0xffffffffu, lead && mine_e->gs < ct0);
      const uint32_t right = __ballot_sync(0xffffffffu, lead && mine_e->ge > ct1) & ~left;
      if (left) open_run[0] = __ffs(left) - 1;
      if (right) open_run[1] = __ffs(right) - 1;
      int unit = 0;                                      // (at most 32 runs of 8 heads)
#pragma unroll 1
      for (uint32_t todo = leads; todo; unit += G) {
        const int first = __ffs(todo) - 1;
        uint32_t members = valid & ~((1u << first) - 1);
        todo &= todo - 1;
        if (todo) members &= (1u << (__ffs(todo) - 1)) - 1;
#pragma unroll 1
        for (int h = (warp + 64 * NW - unit) % NW; h < G; h += NW) {
          float M = -INFINITY, MO = -INFINITY, Ls = 0.f;
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (uint32_t mem = members; mem; mem &= mem - 1) {
            const float* q = entry_part(__ffs(mem) - 1) + G * kPartPitch + 3 * h;
            M = fmaxf(M, q[0]);
            MO = fmaxf(MO, q[2]);
          }
#pragma unroll 1
          for (uint32_t mem = members; mem; mem &= mem - 1) {
            const float* q = entry_part(__ffs(mem) - 1);
            const float4 a = *reinterpret_cast<const float4*>(q + h * kPartPitch + 4 * lane);
            q += G * kPartPitch + 3 * h;
            const float w = ex2_from(q[2], MO);
            Ls += q[1] * ex2_from(q[0], M);
            s.x = fmaf(a.x, w, s.x); s.y = fmaf(a.y, w, s.y);
            s.z = fmaf(a.z, w, s.z); s.w = fmaf(a.w, w, s.w);
          }
          if (first != open_run[0] && first != open_run[1]) {
            const int gd = ent[first].gid, b = small_div(gd, L.Hkv);
            const int64_t head = (int64_t)b * L.Hq + (int64_t)kv_head(L, gd - b * L.Hkv) * G + h;
            const float f = out_factor<KV>(M, MO, Ls);
            uint2 w;
            w.x = pack_bf2(s.x * f, s.y * f);
            w.y = pack_bf2(s.z * f, s.w * f);
            *reinterpret_cast<uint2*>(P.out + head * kD + 4 * lane) = w;
            if (P.lse && lane == 0) P.lse[head] = (M + log2f(Ls)) * 0.6931471805599453f;
          } else {
            float* gp = P.part + (int64_t)((Cfg::kLater ? range : (int)blockIdx.x) * 2 + (first == open_run[0] ? 0 : 1)) * cta_part_floats(G);
            *reinterpret_cast<float4*>(gp + h * kD + 4 * lane) = s;
            if (lane < 3) gp[G * kD + 3 * h + lane] = lane == 0 ? M : lane == 1 ? Ls : MO;
          }
        }
      }
    }
    if (open_run[0] >= 0 || open_run[1] >= 0) {
      __syncthreads();
      // a group that spans ranges c0..c1 counts its arrivals at c0's word, which wraps to zero
      int* finish = reinterpret_cast<int*>(sm + S::kMisc);
      if (tid < 2) {
        const int first = tid ? open_run[1] : open_run[0];
        int last = 0;
        if (first >= 0) {
          const PagedEntry e = ent[first];
          const int c0 = range_of<Cfg::kLater>(split, e.gs), c1 = range_of<Cfg::kLater>(split, e.ge - 1);
          // the CTA's partial before the arrival, the others' after it
          uint32_t old;
          asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;"
                       : "=r"(old) : "l"(P.arrive + c0), "r"((uint32_t)(c1 - c0)) : "memory");
          last = old == (uint32_t)(c1 - c0);
        }
        finish[tid] = last;
      }
      __syncthreads();

      // ---- groups at which this CTA was the last to arrive
      float* wt = reinterpret_cast<float*>(sm + S::kWt);          // [parts][8]
      float* fac = reinterpret_cast<float*>(sm + S::kMisc) + 16;  // [8]
      const int items = G * (kD / 4);
      const int64_t pf = cta_part_floats(G);
      for (int x = 0; x < 2; ++x) {
        if (!finish[x]) continue;
        const PagedEntry e = ent[x ? open_run[1] : open_run[0]];
        const int c0 = range_of<Cfg::kLater>(split, e.gs), np = range_of<Cfg::kLater>(split, e.ge - 1) - c0 + 1;
        // part i: the open end of range c0 + i (its last group for i = 0, its first otherwise)
        const float* part = P.part + (int64_t)c0 * 2 * pf;
        const int b = small_div(e.gid, L.Hkv);
        const int64_t head0 = (int64_t)b * L.Hq + (int64_t)kv_head(L, e.gid - b * L.Hkv) * G;
        // Four channels a thread; where G is small, teams of threads share out the parts.
        // As many parts as the rings hold are copied to shared memory, all copies in flight at once
        // (loads into registers, 8 at a time, took 9 us for 103 parts), while the weights are made.
        const int pb = (int)pf * 4, fit = S::kRing / pb;
        const unsigned char* part_b = reinterpret_cast<const unsigned char*>(part);
        const int teams = NT / items, team = tid / items, it = tid - team * items, h = it >> 5;
        auto copy = [&](int i0, int nb) {                  // a thread copies the 16 bytes it sums up
          if (team < teams)
            for (int i = i0 + team; i < i0 + nb; i += teams)
              cp_async16(sm + (i - i0) * pb + it * 16, part_b + (int64_t)(i * 2 + (i == 0)) * pb + it * 16);
          cp_async_commit();
        };
        copy(0, min(np, fit));
        if (warp < G) {
          // up to 160 parts (all, but for one group over a long line) from registers
          constexpr int kHeld = kPagedMaxCTAs / 32;
          float m[kHeld], l[kHeld], mo[kHeld];
          float M = -INFINITY, MO = -INFINITY, Ls = 0.f;
          auto state = [&](int i) { return part + (i * 2 + (i == 0)) * pf + G * kD + 3 * warp; };
#pragma unroll
          for (int u = 0; u < kHeld; ++u) {
            const int i = lane + 32 * u;
            m[u] = i < np ? __ldcg(state(i)) : -INFINITY;
            l[u] = i < np ? __ldcg(state(i) + 1) : 0.f;
            mo[u] = i < np ? __ldcg(state(i) + 2) : -INFINITY;
          }
#pragma unroll
          for (int u = 0; u < kHeld; ++u) { M = fmaxf(M, m[u]); MO = fmaxf(MO, mo[u]); }
          if (Cfg::kLater)
#pragma unroll 1
            for (int i = lane + 32 * kHeld; i < np; i += 32) {
              M = fmaxf(M, __ldcg(state(i)));
              MO = fmaxf(MO, __ldcg(state(i) + 2));
            }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            MO = fmaxf(MO, __shfl_xor_sync(0xffffffffu, MO, o));
          }
#pragma unroll
          for (int u = 0; u < kHeld; ++u) {
            const int i = lane + 32 * u;
            if (i < np) {
              Ls += l[u] * ex2_from(m[u], M);
              wt[i * 8 + warp] = ex2_from(mo[u], MO);
            }
          }
          if (Cfg::kLater)
#pragma unroll 1
            for (int i = lane + 32 * kHeld; i < np; i += 32) {
              Ls += __ldcg(state(i) + 1) * ex2_from(__ldcg(state(i)), M);
              wt[i * 8 + warp] = ex2_from(__ldcg(state(i) + 2), MO);
            }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) Ls += __shfl_xor_sync(0xffffffffu, Ls, o);
          if (lane == 0) {
            fac[warp] = out_factor<KV>(M, MO, Ls);
            if (P.lse) P.lse[head0 + warp] = (M + log2f(Ls)) * 0.6931471805599453f;
          }
        }
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < np; i0 += fit) {
          if (i0 > 0) {
            __syncthreads();
            copy(i0, min(np - i0, fit));
          }
          cp_async_wait<0>();
          __syncthreads();
          if (team < teams) {
            const int end = min(np, i0 + fit);
#pragma unroll 4
            for (int i = i0 + team; i < end; i += teams) {
              const float4 a = *reinterpret_cast<const float4*>(sm + (i - i0) * pb + it * 16);
              const float w = wt[i * 8 + h];
              s.x = fmaf(a.x, w, s.x); s.y = fmaf(a.y, w, s.y);
              s.z = fmaf(a.z, w, s.z); s.w = fmaf(a.w, w, s.w);
            }
          }
        }
        __syncthreads();
        float4* red = reinterpret_cast<float4*>(sm);
        red[tid] = s;
        __syncthreads();
        if (tid < items) {
          for (int q = 1; q < teams; ++q) {
            const float4 a = red[q * items + it];
            s.x += a.x; s.y += a.y; s.z += a.z; s.w += a.w;
          }
          const float f = fac[h];
          uint2 w;
          w.x = pack_bf2(s.x * f, s.y * f);
          w.y = pack_bf2(s.z * f, s.w * f);
          *reinterpret_cast<uint2*>(P.out + head0 * kD + 4 * it) = w;
        }
        __syncthreads();
      }
    }
    if (!Cfg::kLater || later == 0) return;
    // ---- the next range that nobody has taken; each CTA comes here once too often, so the count
    // wraps to zero
    __syncthreads();                                     // the rings and entries are free
    if (tid == 0) {
      const uint32_t old = atomicInc(P.queue, (uint32_t)(split.n + later - 1));
      *next_range = old < (uint32_t)later ? split.n + (int)old : -1;
    }
    if (tid < 2 * NW) ent[tid].gid = -1;
    __syncthreads();
    range = *next_range;
    if (range < 0) return;
    ct0 = range_start<Cfg::kLater>(split, range);
    ct1 = range_start<Cfg::kLater>(split, range + 1);
  }
}

// ------------------------------------------------------------------ append of new tokens

struct PagedAppendParams {
  PagedPtrs C;
  const uint16_t *k_pre, *v;
  const int32_t *start_pos, *slot_map;
  int64_t n_tok, cap_rows;       // B * n_new; n_pages * page
  int n_new, Hkv;
  uint32_t inv_last;             // 2^16 / (heads of the last block of 8) rounded up: divides exactly
  int step_last;                 // tokens that a CTA copies at once in the last block
  int* status;
  double theta[kD / 2];          // theta_i
  double2 turn[2][kD / 2];       // (cos, sin) of theta_i and of R theta_i
};

// A CTA of 128 threads takes up to 8 KV heads of 2 R consecutive tokens of the flattened
// [B][n_new] axis. Their rows, contiguous in the inputs, are copied to shared memory while the
// angles are made, once for all heads: sin and cos in double of the first token's 64 angles, the
// other tokens of its sequence by turning on (products of cos and sin of theta: off by 2^-50, where
// position * theta itself is rounded by up to 2^-53 of its size). Then half a warp
// per (token, KV head) row, 4 channel pairs a lane, in double. (Eight CTAs an SM, each at another
// of these stages; 256 threads and twice the tokens were 2 to 7 % slower.)
// Bound by HBM: 512 B read, 512 (264) B written per row; bf16 rows run at it (32K tokens of 8 KV
// heads in 43 us in graphs, 45 us in a run of calls, 6.0-6.2 TB/s). e4m3 rows (51 us; 300
// instructions a row pair, 193 for bf16) are bound by the latency of their steps: the issue slots are
// 59 % busy, and the 29 warps an SM has on average wait for results (2.3 cycles an issue), for the
// CTA's barriers (1.8) and for conversions and shared memory (1.7). Single precision with
// carried errors took twice the instructions.
constexpr int kAppendHeads = 8, kAppendThreads = 128;

template <int KV, int R>
__global__ void __launch_bounds__(kAppendThreads, 8)
paged_append_kernel(const __grid_constant__ PagedAppendParams P) {
  constexpr int TOK = 2 * R;
  // (cos, sin) as the lanes read them: [token][channel % 4][channel / 4]; the tokens' K and V rows
  extern __shared__ __align__(16) unsigned char asm_[];
  double2(*ang)[4][16] = reinterpret_cast<double2(*)[4][16]>(asm_);
  unsigned char* rows = asm_ + TOK * 1024;
  __shared__ int32_t slots[TOK];
  const int tid = threadIdx.x, i = tid & 63, sub = tid >> 6;
  const double th = ld_gen(&P.theta[i]);
  const double2 z1 = ld_gen(&P.turn[0][i]), zr = ld_gen(&P.turn[1][i]);
  launch_begin();
  const int64_t tok0 = (int64_t)blockIdx.x * TOK;
  const int g0 = blockIdx.y * kAppendHeads, heads = min(P.Hkv - g0, kAppendHeads);
  const bool last_y = blockIdx.y == gridDim.y - 1;
  int slot = -1;
  if (tid < TOK && tok0 + tid < P.n_tok) slot = P.slot_map[tok0 + tid];
  if (tid < TOK) slots[tid] = slot;
  if (!__syncthreads_or(slot >= 0)) return;            // a CTA of padding
  {
    // a token's K are 16 * heads pieces of 16 bytes, and its V; a pass covers as many whole tokens
    // as there are threads for
    const int u0 = (int)((uint32_t)(tid >> 4) * (last_y ? P.inv_last : 8192u) >> 16);
    const int x = tid - u0 * heads * 16, step = last_y ? P.step_last : 1;
    int64_t src = ((tok0 + u0) * P.Hkv + g0) * kD + x * 8;
    if (u0 < step) {
      uint32_t dst = smem_u32(rows) + u0 * heads * 512 + x * 16;
#pragma unroll 4
      for (int u = u0; u < TOK; u += step, src += step * P.Hkv * kD, dst += step * heads * 512)
        if (slots[u] >= 0) {
          cp_async16_s(dst, P.k_pre + src);
          cp_async16_s(dst + heads * 256, P.v + src);
        }
    }
    cp_async_commit();
  }
  {
    const int64_t b0 = P.n_tok >> 32 ? tok0 / P.n_new : (uint32_t)tok0 / (uint32_t)P.n_new;
    const int64_t j0 = tok0 - b0 * P.n_new;
    int64_t b = b0, j = j0 + sub * R;
    const bool turn = sub > 0 && j < P.n_new;          // the first token's sequence: turned on
    while (j >= P.n_new) { j -= P.n_new; ++b; }
    double2 z = make_double2(1.0, 0.0);
    if (tok0 + sub * R < P.n_tok && !turn) rope_sincos((double)P.start_pos[b] + (double)j, th, &z.y, &z.x);
    if (sub == 0) ang[0][i & 3][i >> 2] = z;
    __syncthreads();
    if (turn) {
      z = ang[0][i & 3][i >> 2];
      z = turned(z, zr);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int u = sub * R + r;
      if (tok0 + u < P.n_tok) {
        if (r > 0) {
          if (++j == P.n_new) {                        // the next sequence begins
            j = 0;
            ++b;
            rope_sincos((double)P.start_pos[b], th, &z.y, &z.x);
          } else {
            z = turned(z, z1);
          }
        }
        if (i == 0 && slots[u] >= 0 && (slots[u] >= P.cap_rows || (int64_t)P.start_pos[b] + j < 0)) {
          set_status(P.status, -6);
          slots[u] = -1;
        }
        if (u > 0) ang[u][i & 3][i >> 2] = z;
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();
  // half a warp stays with its token: 8 / TOK of them share out its heads
  constexpr int kShare = 8 / TOK;
  const int ln = tid & 15, u = (tid >> 4) / kShare;
  slot = slots[u];
  if (slot < 0) return;
  double2 z4[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) z4[e] = ang[u][e][ln];
  const int pid = slot >> P.C.lg;
#pragma unroll 1
  for (int g = (tid >> 4) % kShare; g < heads; g += kShare) {
    const unsigned char* kr = rows + (u * heads * 2 + g) * 256;
    const uint2 a = reinterpret_cast<const uint2*>(kr)[ln];
    const uint2 c = reinterpret_cast<const uint2*>(kr + 128)[ln];
    const uint4 vv = reinterpret_cast<const uint4*>(kr + heads * 256)[ln];
    double kx[8];                                      // channels 4 ln .. 4 ln + 3, their partners
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t wa = e & 2 ? a.y : a.x, wc = e & 2 ? c.y : c.x;
      const double p = e & 1 ? bf_hi(wa) : bf_lo(wa), q = e & 1 ? bf_hi(wc) : bf_lo(wc);
      const double2 z = z4[e];
      kx[e] = p * z.x - q * z.y;
      kx[4 + e] = p * z.y + q * z.x;
    }
    float k[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) k[e] = (float)kx[e];
    const int in = ((g0 + g) << P.C.lg) + (slot & ((1 << P.C.lg) - 1));
    const int64_t row = pid * P.C.page_stride + in;    // below 2^31
    if (KV == kKvBf16) {
      // rounding twice differs from once only where single precision ends up in the middle of two
      // bf16 values (2^-16 of the elements), or has lost a small number's last places
      uint32_t o[4];
      bool unsure = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[e] = pack_bf2(k[2 * e], k[2 * e + 1]);
        unsure = unsure || (__float_as_uint(k[2 * e]) & 0xffffu) == 0x8000u ||
                 (__float_as_uint(k[2 * e + 1]) & 0xffffu) == 0x8000u;
      }
      if (unsure) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = d2bf_rn(kx[2 * e]) | (uint32_t)d2bf_rn(kx[2 * e + 1]) << 16;
      }
      unsigned char* kd = P.C.k + row * 256;
      reinterpret_cast<uint2*>(kd)[ln] = make_uint2(o[0], o[1]);
      reinterpret_cast<uint2*>(kd + 128)[ln] = make_uint2(o[2], o[3]);
      reinterpret_cast<uint4*>(P.C.v + row * 256)[ln] = vv;
    } else {
      float y[8];
      unpack8(vv, y);
      float mk = 0.f, mv = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) { mk = fmaxf(mk, fabsf(k[e])); mv = fmaxf(mv, fabsf(y[e])); }
      // the first step of both maxima in one exchange: even lanes go on with the keys', odd lanes
      // with the values', and divide for them
      const uint32_t team = 0xffffu << (tid & 16);
      float top = fmaxf(ln & 1 ? mv : mk, __shfl_xor_sync(team, ln & 1 ? mk : mv, 1));
#pragma unroll
      for (int o = 2; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(team, top, o));
      const float sc = row_scale(top), inv = __frcp_rn(sc);
      const float sc2 = __shfl_xor_sync(team, sc, 1), inv2 = __shfl_xor_sync(team, inv, 1);
      const uint2 k8 = e4m3_of8(k, ln & 1 ? sc2 : sc, ln & 1 ? inv2 : inv);
      unsigned char* kd = P.C.k + row * 128;
      reinterpret_cast<uint32_t*>(kd)[ln] = k8.x;
      reinterpret_cast<uint32_t*>(kd + 64)[ln] = k8.y;
      reinterpret_cast<uint2*>(P.C.v + row * 128)[ln] = e4m3_of8(y, ln & 1 ? sc : sc2, ln & 1 ? inv : inv2);
      if (ln < 2) (ln ? P.C.vs : P.C.ks)[pid * ((int64_t)P.Hkv << P.C.lg) + in] = sc;
    }
  }
}

// ------------------------------------------------------------------ page reservation

struct PagedReserveParams {
  int32_t *free_pages, *table, *slot_map, *lens_out, *step_lens;
  const int32_t *lens, *new_lens;
  const int64_t* counters;
  int64_t* counters_out;
  int64_t cap;                   // tokens a table row can hold
  int B, n_new, n_pages, stride, lg;
  int* status;
  uint32_t* arrive;
};

constexpr int kResThreads = 512, kResWarps = kResThreads / 32;
constexpr int kResPer = 4096 / kResThreads;        // sequences a thread sums up, at most

// saturating sum of counts (each at most 2^31 - 1)
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return min(a + b, 0x7fffffffu); }

// counter mod n (a 64-bit division only for a counter beyond 2^32)
__device__ __forceinline__ int ring_place(int64_t x, int n) {
  return x >> 32 ? (int)(x % n) : (int)((uint32_t)x % (uint32_t)n);
}

constexpr int kResLittle = 4;                // tokens and page moves that one thread takes on

// One sequence's wish: held and wanted pages. Invalid lengths hold and want nothing.
struct ResWish { int n0, n1, h0, h1; bool bad; };
__device__ __forceinline__ ResWish res_wish(const PagedReserveParams& P, int n0, int n1) {
  ResWish w;
  w.n0 = n0;
  w.n1 = n1;
  w.bad = w.n0 < 0 || w.n1 < 0 || w.n0 > P.cap || w.n1 > P.cap;
  const int64_t r = (1 << P.lg) - 1;
  w.h0 = w.bad ? 0 : (int)((w.n0 + r) >> P.lg);
  w.h1 = w.bad ? 0 : (int)((w.n1 + r) >> P.lg);
  return w;
}
// place i of the ring, i below twice its size
__device__ __forceinline__ int64_t ring_at(const PagedReserveParams& P, int64_t i) {
  return i >= P.n_pages ? i - P.n_pages : i;
}
// One thread's sequence: up to kResLittle page moves and slots. head, tail: its places in the ring.
__device__ __forceinline__ void res_little(const PagedReserveParams& P, int b, int n0, int n1, bool granted,
                                           int64_t head, int64_t tail) {
  const ResWish x = res_wish(P, n0, n1);
  int32_t* row = P.table + (int64_t)b * P.stride;
  int id[kResLittle + 1];                    // the page of the first token, then those taken
  const int pg0 = x.bad ? 0 : x.n0 >> P.lg;
  id[0] = granted && pg0 < x.h0 && P.n_new > 0 ? row[pg0] : 0;
#pragma unroll
  for (int j = 0; j < kResLittle; ++j) {
    if (granted && j < x.h1 - x.h0) {
      id[j + 1] = P.free_pages[ring_at(P, head + j)];
      row[x.h0 + j] = id[j + 1];
    }
    if (granted && j < x.h0 - x.h1) P.free_pages[ring_at(P, tail + j)] = row[x.h1 + j];
  }
#pragma unroll
  for (int j = 0; j < kResLittle; ++j)
    if (j < P.n_new) {
      const int64_t pos = (int64_t)x.n0 + j;
      int slot = -1;
      if (granted && pos < x.n1) {
        const int pg = (int)(pos >> P.lg);
        int pid = id[0];                     // (pages are larger than kResLittle tokens: one or the next)
        if (pg >= x.h0) pid = id[1];
        slot = (pid << P.lg) + (int)(pos & ((1 << P.lg) - 1));
      }
      P.slot_map[(int64_t)b * P.n_new + j] = slot;
    }
}

// Every CTA sums up the whole batch (its lengths come from L2): a thread takes up to 8
// consecutive sequences, one scan over the block. A sequence with little to do (a decode step's:
// a few tokens and pages) is then done by the thread that summed it up. The others are shared out
// among the grid's warps, W / B warps to one, 32 pages at a time: a lane per page loads its id
// (from the ring or the table) once, writes the table entry, and the slots of those pages' tokens
// take the id by a shuffle. Bound by the slot map's bytes for prompts, by the launch and the chain
// of loads (lengths, counters, pages) for a decode step.
// Nothing that a call reads is written before all CTAs have read it: the ring's taken and
// returned entries are disjoint, held table entries are not rewritten, and the lengths and
// counters are written by the CTA that arrives last, so they may be updated in place.
__global__ void __launch_bounds__(kResThreads)
paged_reserve_kernel(const __grid_constant__ PagedReserveParams P) {
  extern __shared__ uint32_t rsm[];
  uint32_t* upto = rsm;                      // [B] pages lacked before each sequence
  uint32_t* back = rsm + P.B;                // [B] pages returned before each sequence
  __shared__ uint32_t wsum[2][kResWarps];
  __shared__ uint32_t s_taken, s_bad, s_last;
  __shared__ int s_hm, s_tm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) { s_taken = 0; s_bad = 0; }
  launch_begin();
  const int64_t head = P.counters[0], tail = P.counters[1];
  const int per = (P.B + kResThreads - 1) / kResThreads, first = tid * per;
  int n0[kResPer], n1[kResPer];
  uint32_t need[kResPer], ret[kResPer], a = 0, c = 0;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kResPer; ++k) {
    n0[k] = n1[k] = 0;
    if (k < per && first + k < P.B) { n0[k] = P.lens[first + k]; n1[k] = P.new_lens[first + k]; }
  }
#pragma unroll
  for (int k = 0; k < kResPer; ++k) {
    const ResWish w = res_wish(P, n0[k], n1[k]);
    need[k] = max(w.h1 - w.h0, 0);
    ret[k] = max(w.h0 - w.h1, 0);
    bad = bad || w.bad;
    a = add_sat(a, need[k]);
    c = add_sat(c, ret[k]);
  }
  uint32_t ia = a, ic = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t ua = __shfl_up_sync(0xffffffffu, ia, o), uc = __shfl_up_sync(0xffffffffu, ic, o);
    if (lane >= o) { ia = add_sat(ia, ua); ic = add_sat(ic, uc); }
  }
  if (lane == 31) { wsum[0][warp] = ia; wsum[1][warp] = ic; }
  // exclusive: the neighbour's inclusive sum (a saturated one cannot be taken apart)
  uint32_t ea = __shfl_up_sync(0xffffffffu, ia, 1), ec = __shfl_up_sync(0xffffffffu, ic, 1);
  if (lane == 0) ea = ec = 0;
  const bool sane = head >= 0 && tail >= head && tail - head <= P.n_pages;
  const uint32_t avail = sane ? (uint32_t)(tail - head) : 0;
  if (warp == kResWarps - 1 && lane < 2)     // the warp with least to do
    (lane ? s_tm : s_hm) = sane ? ring_place(lane ? tail : head, P.n_pages) : 0;
  __syncthreads();
  uint32_t run_c;                            // all returned pages
  {
    uint32_t va = lane < kResWarps ? wsum[0][lane] : 0, vc = lane < kResWarps ? wsum[1][lane] : 0;
#pragma unroll
    for (int o = 1; o < kResWarps; o <<= 1) {
      const uint32_t ua = __shfl_up_sync(0xffffffffu, va, o), uc = __shfl_up_sync(0xffffffffu, vc, o);
      if (lane >= o) { va = add_sat(va, ua); vc = add_sat(vc, uc); }
    }
    run_c = __shfl_sync(0xffffffffu, vc, kResWarps - 1);
    const uint32_t ba = __shfl_sync(0xffffffffu, va, max(warp - 1, 0));
    const uint32_t bc = __shfl_sync(0xffffffffu, vc, max(warp - 1, 0));
    if (warp > 0) { ea = add_sat(ea, ba); ec = add_sat(ec, bc); }
  }
  // more pages than the ring has room for: the lengths or counters are not this pool's
  const bool ok = sane && (int64_t)avail + run_c <= P.n_pages;
  const int hm = s_hm, tm = s_tm;
  const bool few = P.n_new <= kResLittle;
  uint32_t taken = 0, served = 0;            // served: bit k of this thread's sequences
  bool heavy = false;                        // some are left to the warps
#pragma unroll
  for (int k = 0; k < kResPer; ++k) {
    if (k < per && first + k < P.B) {
      const int b = first + k;
      const bool granted = ok && !res_wish(P, n0[k], n1[k]).bad && (need[k] == 0 || add_sat(ea, need[k]) <= avail);
      served |= (uint32_t)granted << k;
      upto[b] = ea;
      back[b] = ec;
      if (need[k] && granted) taken = ea + need[k];
      if (few && need[k] <= kResLittle && ret[k] <= kResLittle) {
        if (blockIdx.x == b % gridDim.x) res_little(P, b, n0[k], n1[k], granted, hm + ea, tm + ec);
      } else {
        heavy = true;
      }
    }
    ea = add_sat(ea, need[k]);
    ec = add_sat(ec, ret[k]);
  }
  taken = __reduce_max_sync(0xffffffffu, taken);
  if (lane == 0 && taken) atomicMax(&s_taken, taken);
  if (bad) s_bad = 1;
  const bool work = __syncthreads_or(heavy);
  if (tid == 0 && blockIdx.x == 0 && (!ok || s_bad)) set_status(P.status, -6);

  if (work) {
    const int W = gridDim.x * kResWarps, share = max(1, W / P.B);     // warps of a sequence
    const int w = blockIdx.x * kResWarps + warp, teams = W / share;
    // a lane loads the lengths of one of this warp's next 32 sequences
    int la = 0, lb = 0, i = 0;
#pragma unroll 1
    for (int b = w / share; b < P.B && w < teams * share; b += teams, ++i) {
      if ((i & 31) == 0 && b + lane * (int64_t)teams < P.B) {
        la = P.lens[b + lane * teams];
        lb = P.new_lens[b + lane * teams];
      }
      const ResWish x = res_wish(P, __shfl_sync(0xffffffffu, la, i & 31), __shfl_sync(0xffffffffu, lb, i & 31));
      if (few && abs(x.h1 - x.h0) <= kResLittle) continue;
      const int64_t u0 = upto[b], r0 = back[b];
      const bool granted = ok && !x.bad && (x.h1 <= x.h0 || u0 + (x.h1 - x.h0) <= avail);
      const int n1 = granted ? x.n1 : x.n0, h1 = granted ? x.h1 : x.h0;
      int32_t* row = P.table + (int64_t)b * P.stride;
      int32_t* slots = P.slot_map + (int64_t)b * P.n_new;
      // pages returned
      for (int j = (w % share) * 32 + lane; j < x.h0 - h1; j += 32 * share)
        P.free_pages[ring_at(P, tm + r0 + j)] = row[h1 + j];
      // pages from the one that the first new token goes to, 32 at a time; then the places of
      // slot_map behind the last page
      const int pg0 = x.bad ? 0 : x.n0 >> P.lg;
      const int chunks = (max(h1 - pg0, 0) + 31) >> 5;
      for (int ch = w % share; ch < chunks; ch += share) {
        const int pg = pg0 + 32 * ch + lane;
        int id = 0;
        if (pg < x.h0) {
          id = row[pg];
        } else if (pg < h1) {
          id = P.free_pages[ring_at(P, hm + u0 + (pg - x.h0))];
          row[pg] = id;
        }
        // tokens of these pages: positions from p0, at least n0
        const int64_t p0 = (int64_t)(pg0 + 32 * ch) << P.lg;
        const int64_t end = min(min(p0 + (32 << P.lg), (int64_t)n1), (int64_t)x.n0 + P.n_new);
        const int64_t start = max(p0, (int64_t)x.n0);
#pragma unroll 4
        for (int64_t p = start; p < end; p += 32) {
          const int64_t pos = p + lane;
          const int pid = __shfl_sync(0xffffffffu, id, (int)(min(pos, end - 1) - p0) >> P.lg);
          if (pos < end) slots[pos - x.n0] = (pid << P.lg) + (int)(pos & ((1 << P.lg) - 1));
        }
      }
      const int got = min(max(n1 - x.n0, 0), P.n_new);
      for (int j = (x.bad ? 0 : got) + (w % share) * 32 + lane; j < P.n_new; j += 32 * share)
        slots[j] = -1;
    }
  }
  // lengths and counters, once every CTA has read them
  __syncthreads();
  if (tid == 0) s_last = gridDim.x == 1 || atomicInc(P.arrive, gridDim.x - 1) == gridDim.x - 1;
  __syncthreads();
  if (!s_last) return;
#pragma unroll
  for (int k = 0; k < kResPer; ++k)
    if (k < per && first + k < P.B) {
      const bool got = (served >> k) & 1u;
      P.lens_out[first + k] = got ? n1[k] : n0[k];
      if (P.step_lens) P.step_lens[first + k] = got && n1[k] > n0[k] ? n1[k] : 0;
    }
  if (tid == 0) {
    P.counters_out[0] = ok ? head + s_taken : head;
    P.counters_out[1] = ok ? tail + run_c : tail;
  }
}

}  // namespace rtp
