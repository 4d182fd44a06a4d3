// Checks the index arithmetic of the row operators and the int8 product
// (moe_rows_index.hpp) on the host: every LDS place, operand and output
// against a model of the buffers, for every tile shape the launch chooses.
#include <cstdio>
#include <cstdlib>
#include <set>
#include <vector>

#include "moe_rows_index.hpp"

static int fails = 0;
#define CHECK(c, ...)                                     \
  do {                                                    \
    if (!(c)) {                                           \
      if (fails++ < 20) {                                 \
        std::printf("line %d: %s: ", __LINE__, #c);       \
        std::printf(__VA_ARGS__);                         \
        std::printf("\n");                                \
      }                                                   \
    }                                                     \
  } while (0)

// LDS of `lines` lines, each place holding line * 8 + chunk, filled by copies 0 .. lines / 8 - 1.
static std::vector<int> copied(int lines) {
  std::vector<int> lds(lines * 8, -1);
  for (int i = 0; i < lines / 8; ++i)
    for (int l = 0; l < 64; ++l) {
      const int line = 8 * i + l / 8, place = i * 64 + l;  // a copy lands at 16 bytes a lane
      CHECK(place < lines * 8 && lds[place] == -1, "copy %d lane %d", i, l);
      lds[place] = line * 8 + moe::chunk_of(i, l);
    }
  for (int r = 0; r < lines; ++r)
    for (int c = 0; c < 8; ++c)
      CHECK(lds[r * 8 + moe::line_place(r, c)] == r * 8 + c, "line %d chunk %d", r, c);
  return lds;
}

// The reads of 64 lanes, 16 lanes an LDS cycle of 256 bytes: no bank group twice.
static void no_conflicts(int (*at)(int, int), int ks) {
  for (int g = 0; g < 4; ++g) {
    std::set<int> banks;
    for (int l = 16 * g; l < 16 * g + 16; ++l) banks.insert(at(l, ks) / 16 % 16);
    CHECK(banks.size() == 16, "quarter %d lanes %d..: %zu of 16 bank groups", ks, 16 * g, banks.size());
  }
}
static int at32(int l, int ks) { return moe::operand32(l, ks); }
static int at16(int l, int ks) { return moe::operand16(l, ks); }

template <int TB, int CB, int WT, int WC, int S>
static void tile() {
  using Sh = moe::TileShape<TB, CB, WT, WC, S>;
  // each wave's copies: a partition of the stage's lines
  std::vector<int> seen(Sh::BM / 8, 0), seenw(Sh::BN / 8, 0);
  for (int w = 0; w < Sh::waves; ++w) {
    for (int j = 0; j < Sh::CPX; ++j) seen.at(Sh::CPX * w + j)++;
    for (int j = 0; j < Sh::CPW; ++j) seenw.at(Sh::CPW * w + j)++;
  }
  for (int v : seen) CHECK(v == 1, "%d", v);
  for (int v : seenw) CHECK(v == 1, "%d", v);
  CHECK(Sh::RING <= 160 * 1024, "%d", Sh::RING);
  const std::vector<int> x = copied(Sh::BM), w = copied(Sh::BN);
  for (int wave = 0; wave < Sh::waves; ++wave) {
    const int wt = wave / WC, wc = wave % WC;
    for (int ks = 0; ks < 4; ++ks)
      for (int l = 0; l < 64; ++l) {
        for (int i = 0; i < TB; ++i) {
          const int at = (wt * TB + i) * 4096 + moe::operand32(l, ks);
          CHECK(at % 16 == 0 && at + 16 <= Sh::XB, "x operand %d", at);
          CHECK(x.at(at / 16) == ((wt * TB + i) * 32 + l % 32) * 8 + 2 * ks + l / 32, "x block %d lane %d", i, l);
        }
        for (int c = 0; c < CB; ++c) {
          const int at = (wc * CB + c) * 4096 + moe::operand32(l, ks);
          CHECK(at + 16 <= Sh::WB, "w operand %d", at);
          CHECK(w.at(at / 16) == ((wc * CB + c) * 32 + l % 32) * 8 + 2 * ks + l / 32, "w block %d lane %d", c, l);
        }
      }
  }
  // epilogue: what a wave stages of a row block, then what it stores
  for (int ES : {2, 4}) {
    const int RB = Sh::row_bytes(ES), STR = Sh::stride(ES);
    std::vector<int> st(32 * STR / ES, -1);
    for (int l = 0; l < 64; ++l)
      for (int c = 0; c < CB; ++c)
        for (int g = 0; g < 4; ++g) {
          const int byte = (l & 31) * STR + 4 * (l >> 5) * ES + (32 * c + 8 * g) * ES;
          CHECK(byte % (4 * ES) == 0, "alignment of %d", byte);
          for (int v = 0; v < 4; ++v) {
            int& e = st.at(byte / ES + v);
            CHECK(e == -1, "written twice");
            e = (l & 31) * 32 * CB + 32 * c + moe::acc_channel(l, 4 * g + v);
          }
        }
    const int LPR = RB / 16, RPI = 64 / LPR;
    std::vector<int> out(32 * 32 * CB, 0);
    for (int q = 0; q < 32 / RPI; ++q)
      for (int l = 0; l < 64; ++l) {
        const int rr = q * RPI + l / LPR, col = l % LPR;
        for (int v = 0; v < 16 / ES; ++v) {
          const int n = col * (16 / ES) + v;
          CHECK(st.at((rr * STR + col * 16) / ES + v) == rr * 32 * CB + n, "row %d channel %d", rr, n);
          out.at(rr * 32 * CB + n)++;
        }
      }
    for (int v : out) CHECK(v == 1, "stored %d times", v);
    CHECK(Sh::waves * 32 * STR <= Sh::RING, "staging %d", Sh::waves * 32 * STR);
  }
}

// k_i8_rows: a wave's stage of 16 TB rows and 16 CB channels.
template <int TB, int CB>
static void rows() {
  const std::vector<int> x = copied(16 * TB), w = copied(16 * CB);
  for (int ks = 0; ks < 2; ++ks)
    for (int l = 0; l < 64; ++l) {
      for (int i = 0; i < TB; ++i)
        CHECK(x.at((2 * i * 1024 + moe::operand16(l, ks)) / 16) == (16 * i + l % 16) * 8 + 4 * ks + l / 16, "x lane %d", l);
      for (int c = 0; c < CB; ++c)
        CHECK(w.at((2 * c * 1024 + moe::operand16(l, ks)) / 16) == (16 * c + l % 16) * 8 + 4 * ks + l / 16, "w lane %d", l);
    }
}

static void norm() {
  for (int m = 8; m <= moe::kNormMaxCols; m += 8) {
    const int V = moe::norm_vecs(m), NT = moe::norm_threads(m);
    CHECK(NT <= 1024 && (NT == 8 || NT == 16 || NT == 32 || NT % 64 == 0), "m %d NT %d", m, NT);
    for (int teams : {moe::norm_fwd_teams(NT), moe::norm_bwd_teams(NT)})
      CHECK(teams >= 1 && NT * teams <= 1024 && (NT * teams) % 64 == 0, "m %d: %d teams of %d", m, teams, NT);
    if (m % 64 && m > 600) continue;  // the columns of some rows
    for (int bf16 = 0; bf16 < 2; ++bf16) {
      std::vector<char> col(m, 0);
      for (int t = 0; t < NT; ++t)
        for (int v = 0; v < V; ++v) {
          const moe::NormCols c = moe::norm_cols(bf16, t, NT, v);
          for (int f : {c.lo, c.hi})
            if (f < m) {
              CHECK(f % 4 == 0 && f + 4 <= m, "m %d column %d", m, f);
              for (int j = 0; j < 4; ++j) col.at(f + j)++;
            }
        }
      for (int i = 0; i < m; ++i) CHECK(col[i] == 1, "m %d column %d: %d times", m, i, col[i]);
    }
  }
  for (int m = 8; m <= 4200; m += 8)  // a row by slabs, and the loads of lanes past its end
    for (int fours = 0; fours < 2; ++fours) {
      std::vector<char> col(m, 0);
      for (int slab = 0; slab < (m + 511) / 512; ++slab)
        for (int lane = 0; lane < 64; ++lane) {
          const moe::NormCols c = moe::slab_cols(fours, lane, slab);
          CHECK(c.lo >= 512 * slab && c.hi + 4 <= 512 * (slab + 1), "slab %d lane %d", slab, lane);
          CHECK(fours || (c.lo % 8 == 0 && c.hi == c.lo + 4 && (c.lo < m) == (c.hi < m)), "slab %d lane %d", slab, lane);
          for (int f : {c.lo, c.hi})
            if (f < m) {
              CHECK(f % 4 == 0 && f + 4 <= m, "m %d column %d", m, f);
              for (int j = 0; j < 4; ++j) col.at(f + j)++;
            }
        }
      for (int i = 0; i < m; ++i) CHECK(col[i] == 1, "m %d column %d: %d times", m, i, col[i]);
    }
  for (int cus : {1, 104, 256, 304})
    for (int m : {8, 64, 256, 512, 1000, 2048, 4096, 8192, 8200, 16384})
      for (int T : {0, 1, 2, 4, 5, 63, 64, 65, 255, 256, 257, 777, 1000, 4097, 100000, 2147483647}) {
        const int b = moe::norm_bwd_blocks(T, m, cus), teams = moe::norm_bwd_teams(moe::norm_threads(m));
        CHECK((T == 0) == (b == 0) && b <= 2 * cus + 4, "T %d m %d: %d blocks", T, m, b);
        CHECK((long long)b * teams < (long long)T + teams || T == 0, "T %d m %d: an empty block of %d", T, m, b);
      }
}

// Each wave's part of the stages, walked from any start, is taken once.
static void walks() {
  for (int lo = 0; lo < 40; lo += 13)
    for (int n = 1; n <= 40; ++n)
      for (int rot = 0; rot < n; ++rot) {
        std::vector<char> seen(n, 0);
        for (int s = lo; s < lo + n; ++s) {
          const int t = moe::turned(s, rot, lo, lo + n);
          CHECK(t >= lo && t < lo + n, "stage %d of %d at %d", t, n, lo);
          seen.at(t - lo)++;
        }
        for (char c : seen) CHECK(c == 1, "a stage of %d taken %d times", n, c);
      }
}

int main() {
  walks();
  for (int ks = 0; ks < 4; ++ks) no_conflicts(at32, ks);
  for (int ks = 0; ks < 2; ++ks) no_conflicts(at16, ks);
  tile<4, 2, 2, 4, 2>();
  tile<2, 2, 2, 4, 3>();
  tile<2, 1, 2, 4, 4>();
  tile<1, 2, 2, 2, 3>();
  tile<1, 2, 1, 4, 2>();
  tile<1, 2, 1, 4, 3>();
  tile<2, 2, 1, 4, 2>();
  tile<2, 2, 1, 4, 3>();
  tile<1, 1, 2, 2, 4>();
  rows<1, 2>();
  rows<4, 2>();
  rows<2, 2>();
  norm();
  if (fails) {
    std::printf("%d failures\n", fails);
    return 1;
  }
  std::printf("rows index check ok\n");
  return 0;
}
