// Gradients of the chunked delta rule (formulas in delta_common.h and below).
#include <type_traits>

#include "delta_common.h"
#include "delta_prep.h"

namespace gdnq {
namespace {

// The workspace goes on with dS' and z of every chunk and head, as the carry
// holds S and w.
__host__ __device__ inline int64_t backward_left_at(const DeltaLaunch& L, int64_t slots) {
  return delta_align(slots * L.H * delta_chunk_bytes(true));
}

// ---------------------------------------------------------------- the chain of dS
//
// As the forward chain, from the last chunk to the first, dS' and z left for the
// gradients as S and w are; bound as it is, by 192 products a chunk.  4 x 8192
// tokens, 16 heads: 590 us.
template <int DK, bool PASS>
__global__ __launch_bounds__(256, 1) void delta_chain_back_kernel(DeltaLaunch L, int row_groups, int64_t left_at) {
  constexpr int KB = DK / 32, TILES = DK / 16, P = PASS ? 2 : 3;  // parts of what passes on
  using Loader = ChainLoader<DK, true>;
  using Buffer = ChainBuffer<DK, true, false>;
  __shared__ __attribute__((aligned(1024))) Buffer buffers[2];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  int within;
  const int unit = xcd_unit(row_groups * (L.H / L.G), within);
  DeltaItem item = delta_item(L, unit / L.G, PASS);
  if (item.b < 0) return;
  item.seg += PASS;  // the segments that another comes before
  const int b = item.b;
  const DeltaSpan s = delta_sequence(L, b);
  const int chunks = (s.tokens + 63) / 64;
  const ChainPlace place = chain_place(L, row_groups, chunks, item, unit % L.G, within);
  const int h = place.h, group = place.group, count = place.end - place.first, last = place.end - 1;
  const int col = group * 64 + wave * 16 + c;
  const bool mine = col < L.dv && !(PASS && place.identity);
  Loader loader;
  loader.init(L, L.dout, h, PASS && place.identity ? 0 : group, wave, lane);

  const int tiles = (L.dk + 31) / 32 * 2;  // of a row of the state that it leaves
  f32x4 S[TILES];  // dS^T
  const int64_t state_row = ((int64_t(b) * L.H + h) * L.dv + col) * L.dk;
  if constexpr (PASS) {
    if (place.identity)
      chain_identity<TILES>(S, col, g);
    else
      chain_load_state<TILES>(S, nullptr, L.dk, col, mine, g);
  } else {
    const float* start = L.dh_last ? L.dh_last + state_row - int64_t(col) * L.dk : nullptr;
    if (place.end < chunks) start = reinterpret_cast<const float*>(delta_segment(L, int(item.at) + item.seg + 1, h));
    chain_load_state<TILES>(S, start, L.dk, col, mine, g);
  }
  loader.clear(buffers[0]);
  loader.clear(buffers[1]);
  if (count > 0)
    loader.template load<true, false>(buffers[0], loader.next(s.first + int64_t(last) * 64, min(64, s.tokens - last * 64), s.slot + last));
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  for (int done = 0; done < count; ++done) {
    const int chunk = last - done;
    const Buffer& buf = buffers[done & 1];
    Buffer& following = buffers[(done + 1) & 1];
    const auto next = loader.next(s.first + int64_t(chunk - 1) * 64, 64, s.slot + chunk - 1);
    const bool paced = chunk > place.first && next.whole;
    if (chunk > place.first && !next.whole) loader.template load<true, false>(following, next);
    auto ahead = [&](auto step) {
      phase();
      if (paced) loader.template step<step.value, false>(following, next);
    };
    float* left = reinterpret_cast<float*>(static_cast<uint8_t*>(L.workspace) + left_at +
                                           ((s.slot + chunk) * L.H + h) * delta_left_bytes(L));
    bf16x8 ring[3][4];
    auto read = [&](auto i) { chain_rows<DK>(buf.k, lane, i.value, ring[i.value % 3]); };
    read(Int<0>{});
    read(Int<1>{});
    phase();
    bf16x8 sp[KB][P];
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      split8(S[2 * j], S[2 * j + 1], sp[j]);
      if (!PASS && mine && j * 32 + g * 8 < L.dk) {
        *reinterpret_cast<f32x4*>(left + left_place(col, 2 * j, tiles, g)) = S[2 * j];
        *reinterpret_cast<f32x4*>(left + left_place(col, 2 * j + 1, tiles, g)) = S[2 * j + 1];
      }
    }
    const float* rows = reinterpret_cast<const float*>(buf.rows);
    auto row4 = [&](int which, int it) { return *reinterpret_cast<const f32x4*>(rows + which * 64 + chain_row(it, g * 4)); };
    phase();
    f32x4 u[4] = {}, tail[4], decay[4];
    bf16x8 m3[P][TRI_BLOCKS], d[2];
    each<KB>([&](auto i) {
      if constexpr (i.value + 2 < KB) read(Int<i.value + 2>{});
      if constexpr (i.value == KB - 2) {
        chain_triangle(buf.tri + TRI_BYTES, lane, m3);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const s16x4 d0 = chain_column(buf.v, 2 * j, wave, lane), d1 = chain_column(buf.v, 2 * j + 1, wave, lane);
          typedef short s16x8 __attribute__((ext_vector_type(8)));
          d[j] = __builtin_bit_cast(bf16x8, s16x8{d0[0], d0[1], d0[2], d0[3], d1[0], d1[1], d1[2], d1[3]});
          if (PASS && place.identity) d[j] = bf16x8{};
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          tail[it] = row4(ROW_TAIL, it);
          decay[it] = row4(ROW_C, it);
        }
      }
      phase();
      const bf16x8(&f)[4] = ring[i.value % 3];
#pragma unroll
      for (int p = P - 1; p >= 0; --p)
#pragma unroll
        for (int it = 0; it < 4; ++it) u[it] = mfma16(f[it], sp[i.value][p], u[it]);
      ahead(Int<i.value>{});  // the loader's first KB steps
    });
    const float whole = rows[ROW_C * 64 + 63];
    bf16x8 kt[2][4][2], dp[2][P], up[2][P], zp[2][P];
    chain_columns<DK>(buf.q, lane, 0, kt[0]);
    phase();
    // transposed triangles: tiles 0 and 1 take both halves of the tokens, 2 and 3 the second
    auto part = [&](f32x4 (&y)[4], const bf16x8 (&m)[TRI_BLOCKS], const bf16x8& x0, const bf16x8& x1) {
#pragma unroll
      for (int it = 0; it < 4; ++it) y[it] = mfma16(m[it < 2 ? it * 2 + 1 : it + 2], x1, y[it]);
#pragma unroll
      for (int it = 0; it < 2; ++it) y[it] = mfma16(m[it * 2], x0, y[it]);
    };
#pragma unroll
    for (int it = 0; it < 4; ++it) u[it] *= tail[it];
#pragma unroll
    for (int p = P - 1; p >= 0; --p) part(u, m3[p], d[0], d[1]);
    // beside these products: c dO in parts
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      f32x4 a, b4;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = decay[2 * j][e] * float(d[j][e]);
        b4[e] = decay[2 * j + 1][e] * float(d[j][4 + e]);
      }
      split8(a, b4, dp[j]);
    }
#pragma unroll
    for (int t = 0; t < TILES; ++t) S[t] *= whole;
    ahead(Int<KB>{});
    phase();
    bf16x8 n2[2][TRI_BLOCKS];
    chain_triangle(buf.tri, lane, n2);
    if constexpr (TILES > 4) chain_columns<DK>(buf.q, lane, 1, kt[1]);
    phase();
    // the part of dS that does not wait for z, half of it while u is split
    chain_update(S, kt[0], dp);
    split8(u[0], u[1], up[0]);
    split8(u[2], u[3], up[1]);
    ahead(Int<KB + 1>{});
    phase();
    chain_columns<DK>(buf.k, lane, 0, kt[0]);
    f32x4 decay_beta[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) decay_beta[it] = row4(ROW_C_BETA, it);
    phase();
    f32x4 z[4] = {};
    part_terms<2, P>([&](auto i, auto j) { part(z, n2[i.value], up[0][j.value], up[1][j.value]); });
    ahead(Int<KB + 2>{});
    if constexpr (TILES > 4) chain_update(S + 4, kt[1], dp);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      split8(z[2 * j] * -decay_beta[2 * j], z[2 * j + 1] * -decay_beta[2 * j + 1], zp[j]);
    ahead(Int<KB + 3>{});
    phase();
    if constexpr (TILES > 4) chain_columns<DK>(buf.k, lane, 1, kt[1]);
    phase();
    chain_update(S, kt[0], zp);
    ahead(Int<KB + 4>{});
    if constexpr (TILES > 4) chain_update(S + 4, kt[1], zp);
    ahead(Int<KB + 5>{});
    static_assert(Loader::LOADS == KB && Loader::STEPS == KB + 6, "every step of the loader is taken");
    phase();
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (!PASS && mine) {
      float* to = left + delta_state_floats(L);
#pragma unroll
      for (int it = 0; it < 4; ++it) *reinterpret_cast<f32x4*>(to + left_place(col, it, 4, g)) = z[it];
    }
  }
  if constexpr (PASS) chain_leave<TILES>(L, item, place, S, col, g);
  if (!PASS && L.dh0 && mine && item.seg == 0) {
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int at = chain_row(t, g * 4);
      if (at < L.dk) *reinterpret_cast<f32x4*>(L.dh0 + state_row + at) = S[t];
    }
  }
}

// ---------------------------------------------------------------- the gradients of a chunk
//
// With S entering, dS' leaving, u = beta w and dx = beta z:
//   dM = dO u^T (j <= i),   dAt = -dx u^T (j < i),   both times rho below
//   dQ = c dO S + dM K
//   dK = dAt K - c dx S + dM^T Q + dAt^T K + (c_64 / c) u dS'
//   d log alpha_t = sum over i >= t > j of dM_ij q_i.k_j + dAt_ij k_i.k_j
//                 + sum over i >= t of q_i.(c dO S)_i - k_i.(c dx S)_i
//                 + sum over j < t of k_j.((c_64 / c) u dS')_j  + c_64 <S, dS'>
// A sum over what passes token t, with nothing subtracted: what lies before or
// behind it wholly is not in it.
//   A workgroup of sixteen waves takes a chunk and key head after another, and
// the key head's value heads in turn (so that their sum needs no atomics and no
// memory): wave (it, quarter) has the 16 tokens of tile it, a quarter of the
// columns (d_k) and half of dM or of dAt.  S, dS', w, z and dO pass through LDS 32
// rows (d_v) at a time, the first four by way of registers, where they are split
// into three parts once for all sixteen waves; the next ones (of the next head, or
// chunk) are loaded while these are used.  Bound by these loads, 208 KB a chunk and
// head at 128 x 128, and the products that they wait for: 16384 tokens, 16 heads take
// 390 us, 1.17 GB at 3.0 TB/s, 22 us a chunk and head on each CU; with two parts,
// loaded as such, it was 316, and dbeta and dlog alpha 4e-6 to 6e-6 of their norm off
// (now 1e-6), more where few large terms cancel.  dQ and dK are formed transposed
// (tokens in lanes), so that a token's factors are a lane's and results leave four at
// a time.
template <int DK>
struct GradientSlab {
  uint8_t states[6][32 * DK * 2], tokens[6][4096];  // S, dS' and w, z, three parts each
};

// Rows of 32 bf16 in LDS.
__device__ __forceinline__ int slab_block(int row, int block) { return row * 64 + ((block ^ (row >> 2 & 3)) << 4); }

// A slab passes through registers, where it is split: four values of S and of dS'
// (with DK 64 in the first eight waves) and of w (waves 0 to 7) or z, loaded while
// the slab before is used.  dO goes straight into LDS.
template <int DK>
struct GradientLoader {
  static constexpr int TILES = DK / 16;
  const uint8_t *left[2], *d, *rows;  // of the carry and the workspace at a chunk and head; dO of its first token; its decays
  int64_t vrow;
  int dk, dv, n, wave, lane, tiles, state_floats;
  bool has_state;
  struct Held {
    f32x4 s, ds, t;
  };
  __device__ __forceinline__ void init(const DeltaLaunch& L, int wave_, int lane_) {
    wave = wave_;
    lane = lane_;
    dk = L.dk;
    dv = L.dv;
    vrow = int64_t(L.H) * L.dv * 2;
    tiles = (dk + 31) / 32 * 2;
    state_floats = int(delta_state_floats(L));
    has_state = wave < 2 * TILES;
  }
  __device__ __forceinline__ void set(const DeltaLaunch& L, int64_t left_at, int64_t slot, int64_t first, int tokens, int h) {
    const int64_t chunk = slot * L.H + h;
    const uint8_t* space = static_cast<const uint8_t*>(L.workspace);
    left[0] = static_cast<const uint8_t*>(L.carry) + chunk * delta_left_bytes(L);
    left[1] = space + left_at + chunk * delta_left_bytes(L);
    rows = space + chunk * delta_chunk_bytes(true) + delta_scalars(true);
    d = static_cast<const uint8_t*>(L.dout) + (first * L.H + h) * int64_t(L.dv) * 2;
    n = tokens;
  }
  // Row of the slab and tile of a wave's values; a lane has columns 4 (lane % 4) .. of
  // the tile (chain_row) in row lane / 4 of the group's.
  __device__ __forceinline__ int state_row() const { return wave / TILES * 16 + (lane >> 2); }
  __device__ __forceinline__ int state_tile() const { return wave % TILES; }
  __device__ __forceinline__ int token_row() const { return (wave >> 2 & 1) * 16 + (lane >> 2); }
  __device__ __forceinline__ bool keep_state(int v0) const {
    return v0 + state_row() < dv && chain_row(state_tile(), (lane & 3) * 4) < dk;
  }
  // From a clamped address where there is nothing: cut to zero in store().
  __device__ __forceinline__ Held load(int v0, uint8_t* outs) const {
    Held x = {};
    if (has_state) {
      const uint32_t at = keep_state(v0) ? uint32_t(((v0 + state_row()) >> 4) * tiles + state_tile()) * 1024 + lane * 16 : lane * 16;
      x.s = *reinterpret_cast<const f32x4*>(left[0] + at);
      x.ds = *reinterpret_cast<const f32x4*>(left[1] + at);
    }
    const uint32_t group = v0 + token_row() < dv ? (v0 + token_row()) >> 4 : 0;
    x.t = *reinterpret_cast<const f32x4*>((wave < 8 ? left[0] : left[1]) + state_floats * 4 + ((group * 4 + (wave & 3)) * 1024 + lane * 16));
    if (wave < 4) {
      const int row = (wave * 64 + lane) / 4, block = (slab_block(row, lane & 3) >> 4) & 3;
      const uint8_t* p = d + row * vrow + (v0 + block * 8) * 2;
      to_lds(row < n && v0 + block * 8 < dv ? p : delta_zeros, outs + wave * 1024);
    }
    return x;
  }
  // Four values, in parts, to their place in each part's matrix.
  __device__ __forceinline__ static void split_to(const f32x4& x, uint8_t* to, int part_bytes) {
    uint32_t a[3], b[3];
    split_pair(f32x2{x[0], x[1]}, a);
    split_pair(f32x2{x[2], x[3]}, b);
#pragma unroll
    for (int p = 0; p < 3; ++p) *reinterpret_cast<uint2*>(to + p * part_bytes) = uint2{a[p], b[p]};
  }
  // The slab into LDS; the sum of this lane's products of S and dS'.
  __device__ __forceinline__ float store(Held x, int v0, GradientSlab<DK>& to) const {
    float sum = 0.0f;
    auto cut = [](bool keep, const f32x4& v) { return __builtin_bit_cast(f32x4, only_if(keep, __builtin_bit_cast(u32x4, v))); };
    if (has_state) {
      const bool keep = keep_state(v0);
      x.s = cut(keep, x.s);
      x.ds = cut(keep, x.ds);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum = fmaf(x.s[e], x.ds[e], sum);
      const int t = state_tile(), at = lds_block<DK>(state_row(), (t >> 1) * 4 + (lane & 3)) + (t & 1) * 8;
      split_to(x.s, to.states[0] + at, sizeof(to.states[0]));
      split_to(x.ds, to.states[3] + at, sizeof(to.states[0]));
    }
    const int t = wave & 3, at = lds_block<64>(token_row(), (t >> 1) * 4 + (lane & 3)) + (t & 1) * 8;
    split_to(cut(v0 + token_row() < dv, x.t), to.tokens[wave < 8 ? 0 : 3] + at, sizeof(to.tokens[0]));
    return sum;
  }
};

// The sum of eight products of values in three parts.
__device__ __forceinline__ float dot8(const bf16x8 (&a)[3], const bf16x8 (&b)[3], float s) {
  part_terms<3, 3>([&](auto i, auto j) {
#pragma unroll
    for (int e = 0; e < 8; e += 2)
      s = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{a[i.value][e], a[i.value][e + 1]}, bf16x2{b[j.value][e], b[j.value][e + 1]}, s, false);
  });
  return s;
}

template <int DK>
__global__ __launch_bounds__(1024) void delta_gradient_kernel(DeltaLaunch L, int64_t left_at, int items) {
  constexpr int KB = DK / 32, TILES = DK / 64;  // tiles of a wave
  constexpr int MAT = 64 * DK * 2;
  static_assert(sizeof(GradientSlab<DK>) >= 4 * 8192, "the triangles take the slab's place");
  __shared__ __attribute__((aligned(1024))) GradientSlab<DK> slab;
  __shared__ __attribute__((aligned(1024))) uint8_t outs[2][4096], ks[MAT], qs[MAT];  // dO of a slab, K, Q
  __shared__ __attribute__((aligned(1024))) float decays[3][512];
  __shared__ float below[2][4][64], row_in[4][64], row_out[4][64], pair_sum[4][64], dots[16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int it = wave >> 2, quarter = wave & 3, kind = quarter >> 1, jt0 = (quarter & 1) * 2;  // kind 0: dM, 1: dAt
  const int share = L.H / L.G;
  const int64_t krow = int64_t(L.G) * L.dk, vrow = int64_t(L.H) * L.dv;
  GradientLoader<DK> loader;
  loader.init(L, wave, lane);
  int c = lane & 15, g = lane >> 4;
  const int col0 = quarter * TILES * 16;  // of the wave's columns

  // Places in LDS.  Blocks are permuted by an exclusive or with bits of the row
  // that 16 rows repeat, so the places of other tiles and blocks are these with
  // constants added (rows) or xored (blocks).
  const int tr_row = g * 8 + (c >> 2), tr_block = (c & 3) >> 1, tr_half = (c & 1) * 8;  // 4 x 16 of a transposing read
  int tr_a = lds_block<DK>(tr_row, quarter * TILES * 2 + tr_block) + tr_half;
  int tr_b = lds_block<DK>(tr_row + 4, quarter * TILES * 2 + tr_block) + tr_half;
  int tr64_a = lds_block<64>(tr_row, tr_block) + tr_half, tr64_b = lds_block<64>(tr_row + 4, tr_block) + tr_half;
  int row_d = lds_block<DK>(c, g), row_64 = lds_block<64>(c, g);  // block g of a tile's row c
  int row_4 = lds_block<DK>(c, quarter * TILES * 2 + (g >> 1)) + (g & 1) * 8;  // four of the wave's columns
  constexpr int TILE_D = 16 * DK * 2, TILE_64 = 16 * 128;  // bytes of a tile's rows
  // What follows from these is formed again in each part of each head: kept, it
  // would not fit the registers, and a reload from memory waits for all the loads
  // into LDS that were made before it.
  auto part = [&] {
    asm volatile("" : "+v"(c), "+v"(g), "+v"(tr_a), "+v"(tr_b), "+v"(tr64_a), "+v"(tr64_b), "+v"(row_d), "+v"(row_64), "+v"(row_4));
  };
  auto columns = [&](const uint8_t* m, int t) { return lds_transposed(m + (tr_a ^ (t << 5)), m + (tr_b ^ (t << 5))); };
  auto columns64 = [&](const uint8_t* m, int tile) { return lds_transposed(m + (tr64_a ^ (tile << 5)), m + (tr64_b ^ (tile << 5))); };

  // the item's slot, key head, first token and tokens; slots without tokens are passed over
  int item = blockIdx.x, n = 0;
  int64_t first = 0;
  auto find = [&](int& i, int64_t& at) {
    int tokens = 0;
    for (; i < items; i += gridDim.x)
      if ((tokens = delta_slot_tokens(L, i / L.G, at)) > 0) break;
    return tokens;
  };
  n = find(item, first);
  // of the decays (the head before's, this one's, the next one's), of dO
  int before = 2, now = 0, turn = 0;
  // d log alpha of the head before, whose sums lie in LDS until the next head's
  // slabs are done: by a wave with the least other work, while slabs are loaded.
  int64_t last_first = 0;
  int last_n = 0, last_h = 0;
  auto finish = [&](const float* row) {
    int l = lane;
    asm volatile("" : "+v"(l));  // or what follows from it is kept in registers through every slab
    // sums over i >= t, and over j < t (not of all up to t less the token's own:
    // its own is far larger where the token forgets much)
    float in = 0.0f, out = 0.0f, all = 0.0f, inside = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      in += row_in[i][63 - l];
      out += l ? row_out[i][l - 1] : 0.0f;
      inside += pair_sum[i][l];
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) all += dots[i];
    in = __shfl(wave_scan_incl(in), 63 - l);
    float da = inside + in + wave_scan_incl(out) + row[ROW_C * 64 + 63] * all;
    if (l < last_n) {
      const int64_t at = (last_first + l) * L.H + last_h;
      if (!L.log_decay) da /= fmaxf(L.alpha[at], 5.42101086e-20f);  // the least decay, 2^-64
      L.dalpha[at] = da;
    }
  };
  typename GradientLoader<DK>::Held held = {};
  if (item < items) {
    loader.set(L, left_at, item / L.G, first, n, item % L.G * share);
    held = loader.load(0, outs[0]);
    if (wave < 2) to_lds(loader.rows, wave * 1024 + lane * 16, decays[0] + wave * 256);
  }
  while (item < items) {
    const int slot = item / L.G, kh = item % L.G;
    int next = item + gridDim.x;
    int64_t next_first = 0;
    const int next_n = find(next, next_first);
    f32x4 dq[TILES] = {}, dk[TILES] = {};
    for (int hs = 0; hs < share; ++hs) {
      const int after = 3 - before - now;
      part();
      int token = it * 16 + c;
      const int h = kh * share + hs;
      const float* row = decays[now];
      f32x4 ds[TILES] = {}, xs[TILES] = {}, ud[TILES] = {};  // dO S, z S, w dS'
      f32x4 pair[2] = {};                                    // dO w^T or z w^T
      float db = 0.0f, dot = 0.0f, bt = 0.0f;
      for (int v0 = 0; v0 < L.dv; v0 += 32, turn ^= 1) {
        asm volatile("s_waitcnt vmcnt(0)" : "+v"(loader.lane) : : "memory");  // with the slab dO and, before the first, the decays
        __syncthreads();  // the slab before, or the triangles, have been read
        dot += loader.store(held, v0, slab);
        // the next slab: of this head, of the next, or of the next chunk
        const bool more = v0 + 32 < L.dv;
        if (!more) {
          if (hs + 1 < share)
            loader.set(L, left_at, slot, first, n, h + 1);
          else if (next < items)
            loader.set(L, left_at, next / L.G, next_first, next_n, next % L.G * share);
          if (wave < 2) to_lds(loader.rows, wave * 1024 + lane * 16, decays[after] + wave * 256);
        }
        held = loader.load(more ? v0 + 32 : 0, outs[turn ^ 1]);  // behind the last chunk the same again
        if (v0 == 0 && hs == 0 && wave < MAT / 1024) {
          const uint8_t* kp = static_cast<const uint8_t*>(L.k) + (first * krow + int64_t(kh) * L.dk) * 2;
          const uint8_t* qp = static_cast<const uint8_t*>(L.q) + (first * krow + int64_t(kh) * L.dk) * 2;
          int r, block;
          lds_place<DK>(wave * 64 + loader.lane, r, block);
          const int64_t at = (r * krow + block * 8) * 2;
          const bool keep = r < n && block * 8 < L.dk;
          to_lds(keep ? kp + at : delta_zeros, ks + wave * 1024);
          to_lds(keep ? qp + at : delta_zeros, qs + wave * 1024);
        }
        __syncthreads();
        if (v0 == 0) {
          if (wave == 3 && last_n > 0) finish(decays[before]);
          bt = row[ROW_BETA * 64 + token];
        }
        auto tokens16 = [&](int part, int tile) { return columns64(slab.tokens[part], tile); };
        const bf16x8 o8 = lds_frag(outs[turn] + it * 1024 + slab_block(c, g));
        {
          const bf16x8 z3[3] = {tokens16(3, it), tokens16(4, it), tokens16(5, it)};
#pragma unroll
          for (int t = 0; t < TILES; ++t) {
            const bf16x8 s3[3] = {columns(slab.states[0], t), columns(slab.states[1], t), columns(slab.states[2], t)};
#pragma unroll
            for (int p = 2; p >= 0; --p) ds[t] = mfma16(s3[p], o8, ds[t]);
            part_terms<3, 3>([&](auto i, auto j) { xs[t] = mfma16(s3[i.value], z3[j.value], xs[t]); });
            phase();
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (jt0 + j > it) continue;
            const bf16x8 w3[3] = {tokens16(0, jt0 + j), tokens16(1, jt0 + j), tokens16(2, jt0 + j)};
            if (kind) {
              part_terms<3, 3>([&](auto i, auto q) { pair[j] = mfma16(z3[i.value], w3[q.value], pair[j]); });
            } else {
#pragma unroll
              for (int p = 2; p >= 0; --p) pair[j] = mfma16(o8, w3[p], pair[j]);
            }
            phase();
          }
          if (quarter == 3) {
            const bf16x8 w3[3] = {tokens16(0, it), tokens16(1, it), tokens16(2, it)};
            db = dot8(w3, z3, db);
            bf16x8 dv8;
#pragma unroll
            for (int e = 0; e < 8; ++e) dv8[e] = bf16(bt * (float(z3[0][e]) + (float(z3[1][e]) + float(z3[2][e]))));
            if (token < n && v0 + g * 8 < L.dv)
              *reinterpret_cast<bf16x8*>(reinterpret_cast<uint8_t*>(static_cast<bf16*>(L.dv_out) + first * vrow + int64_t(h) * L.dv + v0) +
                                         (uint32_t(token) * uint32_t(vrow * 2) + g * 16)) = dv8;
          }
        }
        const bf16x8 w3[3] = {tokens16(0, it), tokens16(1, it), tokens16(2, it)};
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          const bf16x8 d3[3] = {columns(slab.states[3], t), columns(slab.states[4], t), columns(slab.states[5], t)};
          part_terms<3, 3>([&](auto i, auto j) { ud[t] = mfma16(d3[i.value], w3[j.value], ud[t]); });
          phase();
        }
      }
      part();
      token = it * 16 + c;
      uint8_t* pairs = reinterpret_cast<uint8_t*>(&slab);
      if (L.dv <= 32) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // K and Q, for which no other slab has waited
      __syncthreads();
      if (quarter == 3) {
        db = xor32_sum(xor16_sum(db));
        if (token < n && g == 0) L.dbeta[(first + token) * L.H + h] = db;
      }
      dot = wave_allreduce_sum(dot);
      if (lane == 0) dots[wave] = dot;

      // The triangles times rho, in two parts, by columns: row j of `pairs` holds
      // the 64 tokens i.  And what passes each token (sums from the last row up):
      // each element times q.k or k.k, exact products.
      //   rho_ij beta_j = a_i b_j with a_i = 2^(log2 c_i - r), b_j = beta_j 2^(r -
      // log2 c_j); r is that of the row tile's first token, before which the columns
      // of a tile off the diagonal lie, so neither passes 1.
      f32x4 passing[2] = {}, ai = {};
      uint8_t* triangle = pairs + kind * 16384;
      const int* whole = reinterpret_cast<const int*>(row + ROW_WHOLE * 64);
      const float* rest = row + ROW_REST * 64;
      const float rr = rest[it * 16];
      const int rw = whole[it * 16];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = it * 16 + g * 4 + e;
        ai[e] = exp2_difference(rest[i], whole[i], rr, rw);
        if (kind) ai[e] *= -row[ROW_BETA * 64 + i];
      }
#pragma unroll
      for (int jn = 0; jn < 2; ++jn) {
        const int jt = jt0 + jn, j = jt * 16 + c;
        if (jt > (it | 1)) continue;
        float x4[4] = {};
        if (jt <= it) {
          f32x4 xk = {0, 0, 0, 0};
#pragma unroll
          for (int b = 0; b < KB; ++b)
            xk = mfma16(lds_frag((kind ? ks : qs) + it * TILE_D + (row_d ^ (b << 6))), lds_frag(ks + jt * TILE_D + (row_d ^ (b << 6))), xk);
          const float bj = row[ROW_BETA * 64 + j];
          if (jt < it) {
            const float b = bj * exp2_difference(rr, rw, rest[j], whole[j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) x4[e] = ai[e] * b * pair[jn][e];
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = g * 4 + e;
              float rho = bj * exp2_difference(rest[it * 16 + i], whole[it * 16 + i], rest[j], whole[j]);
              if (kind) rho *= -row[ROW_BETA * 64 + it * 16 + i];
              x4[e] = c < i || (c == i && !kind) ? rho * pair[jn][e] : 0.0f;
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) passing[jn][e] = x4[e] * xk[e];
        }
        const int to = jt * TILE_64 + ((lds_block<64>(c, g >> 1) + (g & 1) * 8) ^ (it << 5));
        bf16x4 hi, lo;
        split2(x4, hi, lo);
        *reinterpret_cast<bf16x4*>(triangle + to) = hi;
        *reinterpret_cast<bf16x4*>(triangle + 8192 + to) = lo;
        // sums over the rows from e on, then with those of the lane groups below
#pragma unroll
        for (int e = 2; e >= 0; --e) passing[jn][e] += passing[jn][e + 1];
        const float own = passing[jn][0];
        const float up1 = __shfl_down(own, 16), up2 = __shfl_down(own, 32), up3 = __shfl_down(own, 48);
        const float behind = (g < 3 ? up1 : 0.0f) + (g < 2 ? up2 : 0.0f) + (g < 1 ? up3 : 0.0f);
#pragma unroll
        for (int e = 0; e < 4; ++e) passing[jn][e] += behind;
        if (g == 0) below[kind][it][j] = passing[jn][0];
      }
      part();
      // what the state gives, and its share of the decays' gradient
      {
        const float gm = row[ROW_C * 64 + token], gb = row[ROW_C_BETA * 64 + token], tb = row[ROW_TAIL_BETA * 64 + token];
        float in = 0.0f, out = 0.0f;
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          const int at = it * TILE_D + (row_4 ^ (t << 5));
          const bf16x4 q = *reinterpret_cast<const bf16x4*>(qs + at), k = *reinterpret_cast<const bf16x4*>(ks + at);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = gm * ds[t][e], x = gb * xs[t][e], u = tb * ud[t][e];
            in = fmaf(float(q[e]), a, fmaf(-float(k[e]), x, in));
            out = fmaf(float(k[e]), u, out);
            dq[t][e] += a;
            dk[t][e] += u - x;
          }
        }
        in = xor32_sum(xor16_sum(in));
        out = xor32_sum(xor16_sum(out));
        if (g == 0) row_in[quarter][token] = in, row_out[quarter][token] = out;
      }
      __syncthreads();
      part();
      {
        f32x4 sum = {0, 0, 0, 0};
#pragma unroll
        for (int jn = 0; jn < 2; ++jn) {
          const int jt = jt0 + jn;
          if (jt > it) continue;
          float later = 0.0f;
          for (int i = it + 1; i < 4; ++i) later += below[kind][i][jt * 16 + c];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (jt < it || c < g * 4 + e) sum[e] += passing[jn][e] + later;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum[e] = group_sum<16>(sum[e]);
          if (c == 0) pair_sum[quarter][it * 16 + g * 4 + e] = sum[e];
        }
      }
      part();
      // dM K, dAt K (rows i), dM^T Q, dAt^T K (rows j)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        bf16x8 k8[TILES], q8[TILES];
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          k8[t] = columns(ks + kb * 2 * TILE_D, t);
          q8[t] = columns(qs + kb * 2 * TILE_D, t);
        }
        if (kb <= it / 2) {  // j up to the wave's rows
          const uint8_t* p = pairs + kb * 2 * TILE_64;
          const bf16x8 mh = columns64(p, it), ml = columns64(p + 8192, it), ah = columns64(p + 16384, it), al = columns64(p + 24576, it);
#pragma unroll
          for (int t = 0; t < TILES; ++t) {
            dq[t] = mfma_exact_split(k8[t], mh, ml, dq[t]);
            dk[t] = mfma_exact_split(k8[t], ah, al, dk[t]);
          }
        }
        if (kb >= it / 2) {  // i from the wave's rows on
          const uint8_t* p = pairs + it * TILE_64 + (row_64 ^ (kb << 6));
          const bf16x8 mh = lds_frag(p), ml = lds_frag(p + 8192), ah = lds_frag(p + 16384), al = lds_frag(p + 24576);
#pragma unroll
          for (int t = 0; t < TILES; ++t) {
            dk[t] = mfma_exact_split(q8[t], mh, ml, dk[t]);
            dk[t] = mfma_exact_split(k8[t], ah, al, dk[t]);
          }
        }
      }
      last_first = first;
      last_n = n;
      last_h = h;
      before = now;
      now = after;
    }
    const int token = it * 16 + c;
    if (token < n) {
      bf16* dqp = static_cast<bf16*>(L.dq) + (first + token) * krow + int64_t(kh) * L.dk;
      bf16* dkp = static_cast<bf16*>(L.dk_out) + (first + token) * krow + int64_t(kh) * L.dk;
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        const int at = col0 + t * 16 + g * 4;
        if (at < L.dk) {
          *reinterpret_cast<bf16x4*>(dqp + at) = __builtin_convertvector(dq[t], bf16x4);
          *reinterpret_cast<bf16x4*>(dkp + at) = __builtin_convertvector(dk[t], bf16x4);
        }
      }
    }
    item = next;
    first = next_first;
    n = next_n;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (wave == 3 && last_n > 0) finish(decays[before]);
}

template <int DK>
hipError_t backward(const DeltaLaunch& L, hipStream_t stream) {
  const int64_t slots = delta_slots(L);
  const int64_t left_at = backward_left_at(L, slots);
  if (slots > 0) {
    delta_prep_kernel<DK, true><<<uint32_t(slots * L.H), 256, 0, stream>>>(L);
    if (hipError_t e = hipGetLastError()) return e;
  }
  const int groups = (L.dv + 63) / 64;
  if (L.segments > 1) {
    const int all = groups + (L.dk + 63) / 64;
    delta_chain_back_kernel<DK, true><<<uint32_t(all * L.H * delta_items(L, true)), 256, 0, stream>>>(L, all, left_at);
    if (hipError_t e = hipGetLastError()) return e;
    delta_join_kernel<DK, true><<<uint32_t(groups * L.H * L.B), 256, 0, stream>>>(L, groups);
    if (hipError_t e = hipGetLastError()) return e;
  }
  delta_chain_back_kernel<DK, false><<<uint32_t(groups * L.H * delta_items(L, false)), 256, 0, stream>>>(L, groups, left_at);
  if (hipError_t e = hipGetLastError()) return e;
  const int64_t items = slots * L.G;
  if (items > 0) delta_gradient_kernel<DK><<<uint32_t(items < 256 ? items : 256), 1024, 0, stream>>>(L, left_at, int(items));
  return hipGetLastError();
}

}  // namespace

static DeltaLaunch backward_split(DeltaLaunch L) {
  const int64_t slots = delta_slots(L);
  delta_split(L, backward_left_at(L, slots) + slots * L.H * delta_left_bytes(L));
  return L;
}
size_t delta_backward_workspace_bytes(const DeltaLaunch& L) { return size_t(delta_split_bytes(backward_split(L))); }

hipError_t launch_delta_backward(const DeltaLaunch& L, hipStream_t stream) {
  return L.dk <= 64 ? backward<64>(backward_split(L), stream) : backward<128>(backward_split(L), stream);
}

}  // namespace gdnq
