// Attention over a 4-bit key/value cache for sequences with few rows, gfx950
// (mathematics and operand layouts: kv_tile.h).
//
// Work is counted in steps of a number of keys. A unit -- 16 R rows of one kv
// head of one sequence -- has the steps of the sequence's keys, units follow each
// other by sequence, head and rows, and the steps of the call are shared evenly
// among the workgroups, whatever the lengths. A workgroup finds its share from
// lens and cu alone, so a captured launch follows them. Many sequences are bound
// by the bytes of the keys and values (64 sequences of 1741 to 8192 keys, 64 heads
// over 8 of 128, NVFP4: 368 MB in 66 us, 5.6 TB/s), one by the chain of loads
// before its first keys and after its last (65536 keys: 21 us, 700: 8), rows that
// fill two tiles by the latency of a tile at two waves a SIMD (16 sequences of 4
// tokens, up to 4096 keys, 64 heads over 8: 77 MB in 28 us, 2.7 TB/s).
#include "kv_tile.h"

namespace snip {

namespace {

// Sum over the lanes up to and with each.
__device__ __forceinline__ int wave_prefix(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // the rows before: row_bcast 15, 31
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// Finds the sequence of a step. The sequences are taken in 64 groups of
// neighbours, a group a lane, so that all loads of lens are in flight at once;
// the steps up to and with each group, and with each of 64 sequences of the group
// that was looked into last, lie in the wave's own LDS (registers would cost the
// kernel a wave of occupancy).
struct Cursor {
  int* coarse;                 // [64]
  int* fine;                   // [64]
  int unit_rows, each;         // sequences of a group
  int seq0, before, end;       // the 64 looked into last: the first, the steps before and with them

  __device__ __forceinline__ int cost(const KvAttn& A, int b) const {
    const Span x = span_of(A, b, unit_rows);
    return A.split && prompt_rows(A, x) ? 0 : x.tiles * x.steps * A.c.heads;
  }
  // Steps of all sequences.
  __device__ __forceinline__ int total(const KvAttn& A) {
    const int lane = threadIdx.x & 63;
    each = (A.b.seqs + 63) >> 6;
    int n = 0;
#pragma unroll 4
    for (int j = 0; j < each; ++j) n += cost(A, lane * each + j);
    n = wave_prefix(n);
    coarse[lane] = n;
    before = end = 0;
    __builtin_amdgcn_wave_barrier();
    return __builtin_amdgcn_readlane(n, 63);
  }
  // The sequence that step `at` is in, and the steps before it.
  __device__ __forceinline__ int seek(const KvAttn& A, int at, int* from) {
    const int lane = threadIdx.x & 63;
    if (each > 1 && (at < before || at >= end)) {
      const int g = __ffsll((unsigned long long)__ballot(coarse[lane] > at)) - 1;
      before = g ? __builtin_amdgcn_readfirstlane(coarse[g - 1]) : 0;
      for (int o = 0;; o += 64) {
        seq0 = g * each + o;
        const int n = before + wave_prefix(o + lane < each ? cost(A, seq0 + lane) : 0);
        end = __builtin_amdgcn_readlane(n, 63);
        if (at < end || o + 64 >= each) {
          fine[lane] = n;
          break;
        }
        before = end;
      }
      __builtin_amdgcn_wave_barrier();
    }
    const int* upto = each > 1 ? fine : coarse;
    const int i = __ffsll((unsigned long long)__ballot(upto[lane] > at)) - 1;
    *from = i ? __builtin_amdgcn_readfirstlane(upto[i - 1]) : each > 1 ? before : 0;
    return (each > 1 ? seq0 : 0) + i;
  }
};

// The steps of n workgroups: q each, one more for the first r.
struct Shares {
  uint32_t q, r;
  __device__ __forceinline__ Shares(uint32_t total, uint32_t n) : q(total / n), r(total % n) {}
  __device__ __forceinline__ int first(uint32_t w) const { return (int)(w * q + (w < r ? w : r)); }
  __device__ __forceinline__ int owner(uint32_t at) const {   // of a step
    const uint32_t many = r * (q + 1);
    return (int)(at < many ? at / (q + 1) : r + (at - many) / q);
  }
};

}  // namespace

// What a workgroup leaves for the joining launch: two slots, of the unit that
// its share begins within and of the one that it ends within (maxima, sums and
// rows of output), and where the latter's output belongs.
struct Left {
  int64_t row0;                // first row of the sequence
  int rows, r0, head;          // rows of the unit (0: none is left), its first, its kv head
  int last;                    // the workgroup that has the unit's last step
};

namespace {

constexpr int slot_floats(int dim, int rows) { return rows * (dim + 2); }

// Row tiles of a unit: two decode a key once for up to 32 rows, at the price of a
// wave of occupancy (16 sequences of 4 tokens, 64 heads over 8: 34 us, with one
// tile 36; 8 of 32 tokens: 82 and 126). Waves of a SIMD that the registers are
// held to, and workgroups: as many as are resident.
constexpr int most_tiles(int dim) { return dim == 256 ? 1 : 2; }
constexpr int waves_of(int dim, int tiles) { return dim == 256 ? 2 : (dim == 128 ? 3 : 4) - (tiles == 2); }
constexpr int workers_of(int dim, int tiles) { return 256 * waves_of(dim, tiles); }

template <int E>
__device__ __forceinline__ void store_few(void* p, bool f32, int64_t off, const float (&x)[E]) {
  if constexpr (E == 2) {
    if (f32)
      *reinterpret_cast<float2*>(static_cast<float*>(p) + off) = make_float2(x[0], x[1]);
    else
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p) + off) = pack_bf16(x[0], x[1]);
  } else {
    store_whole(p, f32, off, x);
  }
}

template <int FMT, int D, int NR, int kWaves, bool NT>
__global__ __launch_bounds__(64 * kWaves, waves_of(D, NR)) void kv_attn_kernel(KvAttn A) {
  using G = Geo<FMT, D>;
  constexpr int LD = D + 4;                            // a row in LDS: the lanes' rows meet different banks
  constexpr int kKeys = 32 * kWaves;                   // of a round of the waves
  constexpr int kUnit = kRows * NR;
  __shared__ float stats[2][kWaves][kRows];
  __shared__ f4_t part[kWaves][kRows * LD / 4];
  __shared__ int upto[kWaves][2][64];
  const int lane = threadIdx.x & 63, n = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ek = G::NV ? entries(A.c.texp)[0] : 0, ev = G::NV ? entries(A.c.texp)[1] : 0;
  Cursor cur;
  cur.coarse = upto[wave][0];
  cur.fine = upto[wave][1];
  cur.unit_rows = kUnit;
  const Shares shares(A.each ? A.each * A.b.seqs : cur.total(A), gridDim.x);
  int at = shares.first(blockIdx.x);
  const int stop = shares.first(blockIdx.x + 1);
  if (at >= stop) {
    if (A.left && threadIdx.x == 0) A.left[blockIdx.x] = Left{0, 0, 0, 0, 0};
    return;
  }

  // A share's part of a unit. Its queries and first keys are asked for before the
  // one before it is joined.
  struct Part {
    int64_t row0, pos0;
    int seq, head, r0, rows;
    int begin, last;           // keys
    bool all, goes_on;         // the whole unit; a unit that an earlier workgroup began
    int owner;                 // of the unit's last step
  };
  Rows<FMT, D> R[NR];
  Tile<FMT, D> T0, T1;
  struct Pages {
    int p[2];
  };
  Pages g0, g1;
  auto setup = [&](Part& P) {
    int from;
    if (A.each) {
      P.seq = at / A.each;
      from = P.seq * A.each;
    } else {
      P.seq = cur.seek(A, at, &from);
    }
    const Span U = span_of(A, P.seq, kUnit);
    const int unit = A.each ? at - from : (at - from) / U.steps, s0 = A.each ? 0 : (at - from) % U.steps;
    const int s1 = stop - at < U.steps - s0 ? s0 + (stop - at) : U.steps;
    at += s1 - s0;
    P.row0 = U.row0;
    P.pos0 = U.pos0;
    P.head = unit / U.tiles;
    P.r0 = unit % U.tiles * kUnit;
    P.rows = U.rows - P.r0 < kUnit ? U.rows - P.r0 : kUnit;
    const int64_t begin = (int64_t)(first_key(A, U.pos0) & ~31) + (int64_t)s0 * A.step, end = begin + (int64_t)(s1 - s0) * A.step - 1;
    const int unit_last = limit(A, U.pos0 + (P.r0 + P.rows - 1) / A.group);
    P.begin = (int)begin;
    P.last = end < unit_last ? (int)end : unit_last;
    P.all = s1 - s0 == U.steps;
    P.goes_on = s0 > 0;
    P.owner = P.all ? 0 : shares.owner(at - s1 + U.steps - 1);
  };
  // The table's entries are asked for two rounds ahead.
  auto pages = [&](const Part& P, int key) {
    const Entries table = entries(A.b.table + (int64_t)P.seq * A.b.table_ld);
    Pages g;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = key + 16 * h < P.last ? key + 16 * h : P.last;
      g.p[h] = table[(k > 0 ? k : 0) >> A.c.shift];
    }
    return g;
  };
  auto mapped = [&](const Pages& g, int h) { return (uint32_t)g.p[h] < (uint32_t)A.c.pages; };
  // Loads are never skipped, since the wait for a tile counts those of the next
  // one: beyond the last key, and where a page is not mapped, they read others.
  auto load = [&](const Part& P, int key, const Pages& g, Tile<FMT, D>& T) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      load_half<FMT, D, NT>(A.c, kv_slot(A.c, mapped(g, h) ? g.p[h] : 0, P.head, (key + 16 * h) & ((1 << A.c.shift) - 1)), T.k[h],
                        T.ks[h], T.v[h], T.vs[h]);
  };
  auto issue = [&](const Part& P) {
    const int key = P.begin + 32 * wave;
    g0 = pages(P, key);
    g1 = pages(P, key + kKeys);
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int r = P.r0 + kRows * i + n;
      R[i].load(kRows * i + n < P.rows
                    ? A.q + (P.row0 + r / A.group) * A.ldq + (int64_t)(P.head * A.group + r % A.group) * D
                    : nullptr);
    }
    load(P, key, g0, T0);
  };

  Left left = {0, 0, 0, 0, 0};
  Part P;
  setup(P);
  issue(P);
  while (true) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int r = kRows * i + n;
      const int64_t pos = P.pos0 + (P.r0 + r) / A.group;
      R[i].start(A.scale, ek);
      R[i].last = r < P.rows ? limit(A, pos) : -1;
      R[i].first = first_key(A, pos);
    }
    // keys of any row of the unit, and of all
    const int64_t p0 = P.pos0 + P.r0 / A.group, p1 = P.pos0 + (P.r0 + P.rows - 1) / A.group;
    const int first = first_key(A, p0), every_first = first_key(A, p1), every_last = limit(A, p0), last = P.last;
    auto use = [&](int key, const Pages& g, Tile<FMT, D>& T) {
      // scores: s[i][h][j] is key 16 h + 4 c + j for row n of tile i
      f4_t s[NR][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < NR; ++i) s[i][h] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int l = 0; l < G::KL; ++l) {
          h2_t sc = {};
          float e = 0.0f;
          if constexpr (G::NV)
            sc = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(T.ks[h][l], 1.0f, false);
          else
            e = e8m0_val(T.ks[h][l]);
#pragma unroll
          for (int w = 0; w < G::KD; ++w) {
            const int b = G::SB == 2 ? w / 2 : 0;      // block of the piece
            const u32x4_t k = decode_key<FMT>(T.k[h][l][w], h2_t{sc[b], sc[b]}, e);
#pragma unroll
            for (int i = 0; i < NR; ++i) s[i][h] = mfma<FMT>(k, R[i].q[l][w], s[i][h]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][h][j] *= R[i].factor;
      const bool whole = mapped(g, 0) & mapped(g, 1) & (key >= every_first) & (key + 31 <= every_last);
      if (!whole) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k0 = key + 16 * h + 4 * c, end = mapped(g, h) ? last : -1;
          uint32_t keep = 0u;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int i = 0; i < NR; ++i)
              s[i][h][j] = ((k0 + j >= R[i].first) & (k0 + j <= R[i].last) & (k0 + j <= end)) ? s[i][h][j] : -__builtin_inff();
            keep |= ((k0 + j >= first) & (k0 + j <= end)) ? 0xFFu << (8 * j) : 0u;
          }
          // values of places that no row sees may be anything: their scales are replaced
#pragma unroll
          for (int l = 0; l < G::VL; ++l) T.vs[h][l] &= keep;
        }
      }
      float top[NR];
      bool above = false;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        top[i] = kLowest;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) top[i] = fmaxf(top[i], s[i][h][j]);
        above |= top[i] > R[i].m + (kLag + kLift<FMT>);
      }
      if (__any(above)) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const float m = fmaxf(row_max(top[i]) - kLift<FMT>, R[i].m), f = __builtin_amdgcn_exp2f(R[i].m - m);
          R[i].m = m;
          R[i].l *= f;
#pragma unroll
          for (int d = 0; d < G::DT; ++d) R[i].o[d] *= f;
        }
      }
      u32x4_t ph[NR], pl[NR];                          // fp16, or the two parts in bf16
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          p[j] = __builtin_amdgcn_exp2f(s[i][j / 4][j % 4] - R[i].m);
          R[i].l += p[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (G::NV) {
            ph[i][j] = bits(h2_t{(_Float16)p[2 * j], (_Float16)p[2 * j + 1]});
          } else {
            ph[i][j] = pack_bf16(p[2 * j], p[2 * j + 1]);
            pl[i][j] = pack_bf16(p[2 * j] - bf16_lo(ph[i][j]), p[2 * j + 1] - bf16_hi(ph[i][j]));
          }
        }
      }
#pragma unroll
      for (int l = 0; l < G::VL; ++l) {
        uint32_t v0[2 * G::VB][2], v1[2 * G::VB][2];
        decode_values<FMT, D>(T.v[0][l], T.vs[0][l], v0);
        decode_values<FMT, D>(T.v[1][l], T.vs[1][l], v1);
#pragma unroll
        for (int d = 0; d < 2 * G::VB; ++d) {
          const u32x4_t a = {v0[d][0], v0[d][1], v1[d][0], v1[d][1]};
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            f4_t& o = R[i].o[l * 2 * G::VB + d];
            o = mfma<FMT>(a, ph[i], o);
            if constexpr (!G::NV) o = mfma<FMT>(a, pl[i], o);
          }
        }
      }
    };

    int key = P.begin + 32 * wave;
    if (key <= last) {
      while (true) {
        load(P, key + kKeys, g1, T1);
        const Pages g2 = pages(P, key + 2 * kKeys);
        use(key, g0, T0);
        key += kKeys;
        if (key > last) break;
        load(P, key + kKeys, g2, T0);
        const Pages g3 = pages(P, key + 2 * kKeys);
        use(key, g1, T1);
        key += kKeys;
        if (key > last) break;
        g0 = g2;
        g1 = g3;
      }
    }
    const bool more = at < stop;
    Part N = P;
    if (more) {
      setup(N);
      issue(N);
    }

    // the waves' shares of the rows, joined, a tile at a time: the unit's output, or one of the workgroup's two slots
    float* slot = A.part + (2 * (int64_t)blockIdx.x + !P.goes_on) * slot_floats(D, kUnit);
    if (!P.all && !P.goes_on) left = Left{P.row0, P.rows, P.r0, P.head, P.owner};
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      if (kRows * i >= P.rows) break;
      const float l = row_sum(R[i].l);
      if (c == 0) {
        stats[0][wave][n] = R[i].m;
        stats[1][wave][n] = l;
      }
#pragma unroll
      for (int v = 0; v < G::VL; ++v)
#pragma unroll
        for (int j = 0; j < 4; ++j)                    // O^T's row 4 c + j in 2 VB tiles: dimensions in a row
#pragma unroll
          for (int d = 0; d < 2 * G::VB; d += 4)
            part[wave][(n * LD + v * 32 * G::VB + (4 * c + j) * 2 * G::VB + d) / 4] =
                f4_t{R[i].o[v * 2 * G::VB + d][j], R[i].o[v * 2 * G::VB + d + 1][j], R[i].o[v * 2 * G::VB + d + 2][j], R[i].o[v * 2 * G::VB + d + 3][j]};
      __syncthreads();
      constexpr int LR = 4 * kWaves;                   // lanes of a row
      constexpr int E = D / LR < 4 ? D / LR : 4;
      const int row = threadIdx.x / LR, d0 = threadIdx.x % LR * (D / LR);
      float M = kLowest, L = 0.0f, w[kWaves];
#pragma unroll
      for (int k = 0; k < kWaves; ++k) M = fmaxf(M, stats[0][k][row]);
#pragma unroll
      for (int k = 0; k < kWaves; ++k) {
        w[k] = __builtin_amdgcn_exp2f(stats[0][k][row] - M);
        L += stats[1][k][row] * w[k];
      }
      const int ur = kRows * i + row;
      if (ur < P.rows) {
        const int rr = P.r0 + ur;
        const int64_t t = P.row0 + rr / A.group;
        const int qh = P.head * A.group + rr % A.group;
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
        for (int d = 0; d < D / LR; d += E) {
          float x[E];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            x[e] = 0.0f;
#pragma unroll
            for (int k = 0; k < kWaves; ++k) x[e] += reinterpret_cast<const float*>(part[k])[row * LD + d0 + d + e] * w[k];
            if (P.all) x[e] = output<FMT>(x[e], inv, ev);
          }
          if (P.all)
            store_few(A.out, false, t * A.ldo + (int64_t)qh * D + d0 + d, x);
          else
            store_few(slot, true, 2 * kUnit + ur * D + d0 + d, x);
        }
        if (d0 == 0) {
          if (!P.all) {
            slot[ur] = M;
            slot[kUnit + ur] = L;
          } else if (A.lse) {
            store_lse(A, t, qh, M, L);
          }
        }
      }
      if (i + 1 < NR || more) __syncthreads();
    }
    if (!more) break;
    P = N;
  }
  if (A.left && threadIdx.x == 0) A.left[blockIdx.x] = left;
}

// A unit that several workgroups had a share of, joined: blockIdx.x is the one
// that has its first step, blockIdx.y the row. The parts are taken by several
// groups of lanes and added in a fixed order.
template <int FMT, int D, int NR>
__global__ __launch_bounds__(256) void kv_join_kernel(KvAttn A) {
  constexpr int LR = D / 4, SUBS = 256 / LR;           // lanes of a row, parts taken at once
  constexpr int kUnit = kRows * NR;
  __shared__ float sm[SUBS], sl[SUBS];
  __shared__ f4_t so[SUBS][LR];
  const int w0 = blockIdx.x, row = blockIdx.y;
  const Left U = A.left[w0];
  if (row >= U.rows) return;
  const int w1 = U.last;
  auto slot = [&](int w) { return A.part + (2 * (int64_t)w + (w == w0)) * slot_floats(D, kUnit); };
  const int sub = threadIdx.x / LR, d = threadIdx.x % LR * 4;
  float M = kLowest, L = 0.0f;
  f4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
  if (w1 - w0 < SUBS) {
    if (w0 + sub <= w1) {
      const float* p = slot(w0 + sub);
      M = p[row];
      L = p[kUnit + row];
      x = *reinterpret_cast<const f4_t*>(p + 2 * kUnit + row * D + d);
    }
  } else {
    for (int w = w0 + sub; w <= w1; w += 4 * SUBS) {   // four parts in flight
      f4_t v[4];
      float m[4], l[4], top = M;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool in = w + u * SUBS <= w1;
        const float* p = slot(in ? w + u * SUBS : w);
        m[u] = in ? p[row] : kLowest;
        l[u] = in ? p[kUnit + row] : 0.0f;
        v[u] = *reinterpret_cast<const f4_t*>(p + 2 * kUnit + row * D + d);
        if (!in) v[u] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) top = fmaxf(top, m[u]);
      const float old = __builtin_amdgcn_exp2f(M - top);
      M = top;
      L *= old;
      x *= old;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float f = __builtin_amdgcn_exp2f(m[u] - M);
        L += l[u] * f;
        x += v[u] * f;
      }
    }
  }
  so[sub][threadIdx.x % LR] = x;
  if (d == 0) {
    sm[sub] = M;
    sl[sub] = L;
  }
  __syncthreads();
  if (sub) return;
  M = kLowest;
  L = 0.0f;
  x = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < SUBS; ++i) M = fmaxf(M, sm[i]);
#pragma unroll
  for (int i = 0; i < SUBS; ++i) {
    const float f = __builtin_amdgcn_exp2f(sm[i] - M);
    L += sl[i] * f;
    x += so[i][threadIdx.x] * f;
  }
  const int rr = U.r0 + row;
  const int64_t t = U.row0 + rr / A.group;
  const int qh = U.head * A.group + rr % A.group;
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  const int ev = FMT == SNIP_NVFP4 ? A.c.texp[1] : 0;
  const float y[4] = {output<FMT>(x[0], inv, ev), output<FMT>(x[1], inv, ev), output<FMT>(x[2], inv, ev), output<FMT>(x[3], inv, ev)};
  store_whole(A.out, false, t * A.ldo + (int64_t)qh * D + d, y);
  if (A.lse && d == 0) store_lse(A, t, qh, M, L);
}

// Keys up to which a workgroup takes a unit as a whole: the second launch costs
// as much as five rounds of eight waves (64 sequences of 1024 tokens, 8 kv heads
// of 128: 17 us, shared and joined 28; one sequence 10.0 and 10.6).
constexpr int kShort = 1280;
// Bytes of a cache from which it is read past the last-level cache, where it
// cannot stay (362 MB: 82 -> 74 us; 75 MB, read again and again: 28 -> 30).
constexpr int64_t kStream = (int64_t)128 << 20;
// Mean rows of a sequence from which a call is one of prompts; rows of a sequence
// up to which it is left to this file's launch all the same: a token's heads, and
// with more than kFar keys kSome. Such rows follow the prompts in a launch of their
// own, 5 us with few keys; among the prompts, whose units are not split over keys,
// one unit with many keys outlasts the rest. 64 heads over 8 of 128, us, kSome rows
// left to this launch and not:
//     2048 tokens and 4 after   512: 115, 110   1024: 109, 116   2048: 109, 142   4096: 109, 196   65536: 143, 1936
//     64 sequences of 1 to 33 new tokens, up to 2048 keys: 126, 120; 16 of 2 to 64, up to 4096: 138, 132
// With kFar both of the latter are at 120 and 132.
constexpr int kPrompt = 64, kFew = 16, kSome = 64, kFar = 1024;

}  // namespace

int64_t kv_attn_tiles(int64_t tokens, int64_t seqs, int64_t group) { return tokens * group / kRows + seqs; }

size_t kv_attn_slots(int dim) {
  size_t most = 0;
  for (int t = 1; t <= most_tiles(dim); ++t) {
    const size_t n = (size_t)workers_of(dim, t) * (2 * slot_floats(dim, kRows * t) * sizeof(float) + sizeof(Left));
    most = n > most ? n : most;
  }
  return most;
}

KvPlan kv_attn_plan(int format, int dim, KvAttn* a) {
  KvPlan p = {};
  const KvBatch& b = a->b;
  // units of `rows` rows, of all kv heads, at most
  auto units = [&](int rows) {
    return (b.cu ? a->tokens * a->group / rows + b.seqs : (int64_t)b.seqs * ((a->group + rows - 1) / rows)) * a->c.heads;
  };
  // Prompts: rows enough for a sequence's decoding to be shared, and units enough
  // to fill the GPU, since a unit is not split (8 sequences of 32 tokens after
  // 8192, 64 heads over 8: 128 units).
  const int64_t mean = a->tokens * a->group / b.seqs;
  const int unit = kv_prompt_rows(dim);
  const int64_t full = a->tokens * a->group / unit * a->c.heads;
  p.prompt = mean >= kPrompt && full >= 256 && units(unit) < (1 << 24);
  p.prompt_waves = dim < 256 && full < 1024 ? 8 : 4;     // measured at kv_prompt_kernel
  p.prompt_wg = p.prompt ? (unsigned)units(unit) : 0;
  a->split = p.prompt && b.seqs > 1;
  a->few = a->split ? kFew : 0;
  a->some = a->split ? kSome : 0;
  a->far = kFar;
  p.few = !p.prompt || a->split;
  const bool whole = b.max_len <= kShort && !p.prompt;
  p.join = p.few && !whole;
  p.wide = whole && units(kRows) <= 256;                 // no more than CUs (512: 21 us, with four waves 17)
  p.two = most_tiles(dim) > 1 && mean > kRows && !p.wide && !a->split;
  const int tiles = p.two ? 2 : 1, block = format == SNIP_NVFP4 ? 16 : 32;
  const int64_t each = units(kRows * tiles);
  // Whole units: more than are resident, which evens the lengths out, but not a
  // workgroup each where there are many (256 sequences of 1200 tokens, 2048 units:
  // 79 us, of 256 to 512: 38, and 77 and 36 with twice as many as are resident).
  const int64_t workers = workers_of(dim, tiles);
  p.few_wg = (unsigned)(!whole ? workers : each < 2 * workers ? each : 2 * workers);
  p.join_rows = !b.cu && a->group < kRows * tiles ? a->group : kRows * tiles;
  p.past = !whole && (((int64_t)a->c.pages * a->c.heads) << a->c.shift) * (dim + 2 * dim / block) >= kStream;
  // Steps are counted in 31 bits, whatever the lengths that the tables allow.
  a->step = 32 * kWaves;
  while (a->step < b.max_len && (whole || (double)each * ((double)b.max_len / a->step + 1.0) >= 2147483647.0)) a->step *= 2;
  // A token each and units of one step: no search by lens (16 keys: 6.7 -> 6.2 us, 256 sequences of 256 to 512: 41 -> 38)
  a->each = whole && !b.cu ? (a->group + kRows * tiles - 1) / (kRows * tiles) * a->c.heads : 0;
  a->left = p.join ? reinterpret_cast<Left*>(a->part + (size_t)workers_of(dim, tiles) * 2 * slot_floats(dim, kRows * tiles)) : nullptr;
  return p;
}

hipError_t launch_kv_few(int format, int dim, const KvPlan& p, const KvAttn& a, hipStream_t s) {
  return kv_dispatch(format, dim, [&](auto f, auto d) {
    constexpr int FMT = decltype(f)::value, D = decltype(d)::value;
    auto go = [&](auto t) {
      constexpr int NR = decltype(t)::value;
      if (p.past)
        kv_attn_kernel<FMT, D, NR, kWaves, true><<<p.few_wg, 64 * kWaves, 0, s>>>(a);
      else
        kv_attn_kernel<FMT, D, NR, kWaves, false><<<p.few_wg, 64 * kWaves, 0, s>>>(a);
    };
    if (p.wide)
      kv_attn_kernel<FMT, D, 1, 8, false><<<p.few_wg, 64 * 8, 0, s>>>(a);
    else if (p.two)
      go(std::integral_constant<int, most_tiles(D)>{});
    else
      go(std::integral_constant<int, 1>{});
    return hipGetLastError();
  });
}

hipError_t launch_kv_join(int format, int dim, const KvPlan& p, const KvAttn& a, hipStream_t s) {
  return kv_dispatch(format, dim, [&](auto f, auto d) {
    constexpr int FMT = decltype(f)::value, D = decltype(d)::value;
    const dim3 grid(p.few_wg - 1, p.join_rows);
    if (p.two)
      kv_join_kernel<FMT, D, most_tiles(D)><<<grid, 256, 0, s>>>(a);
    else
      kv_join_kernel<FMT, D, 1><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
  });
}

}  // namespace snip
