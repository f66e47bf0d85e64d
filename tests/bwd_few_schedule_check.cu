// Host-only check of the few-row order of the backward's units (rlk_bwd.cuh), run by
// tests/test_bwd_few_schedule.py on the CPU: every unit appears exactly once, with
// and without dW; every dHidden and dW unit comes after the recompute units it
// waits for; every tile stays inside the chunk's columns of the dX matrix.  Prints
// "OK <units>" or the first violation.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <tuple>

#include "rlk_bwd.cuh"

using namespace rlk;

int main(int argc, char** argv) {
  if (argc != 5) return 2;
  const long long T = atoll(argv[1]), H = atoll(argv[2]), V = atoll(argv[3]), ldx = atoll(argv[4]);
  long long total = 0;
  for (int with_dw = 0; with_dw < 2; ++with_dw) {
    const BwdPlan P = make_bwd_plan(T, H, V, ldx, with_dw != 0, true);
    std::map<std::tuple<int, int, int, int>, long long> index;
    for (long long u = 0; u < P.total; ++u) {
      const BwdUnit x = bwd_decode(P, static_cast<int>(u));
      if (x.type < 0 || x.c < 0 || x.c >= P.NC) { printf("BAD decode at %lld\n", u); return 1; }
      if (!index.emplace(std::make_tuple(x.type, x.c, x.a, x.b), u).second) {
        printf("DUP unit at %lld\n", u);
        return 1;
      }
    }
    if (bwd_decode(P, static_cast<int>(P.total)).type >= 0) { printf("unit past the end\n"); return 1; }
    long long expect = 0;
    for (int c = 0; c < P.NC; ++c) expect += bwd_nR(P, c) + bwd_nH(P) + (with_dw ? bwd_nD(P, c) : 0);
    if (expect != P.total) { printf("COUNT %lld vs %lld\n", expect, P.total); return 1; }
    auto at = [&](int t, int c, int a, int b) -> long long {
      auto it = index.find(std::make_tuple(t, c, a, b));
      return it == index.end() ? -1 : it->second;
    };
    for (auto& kv : index) {
      const int t = std::get<0>(kv.first), c = std::get<1>(kv.first);
      const int a = std::get<2>(kv.first), b = std::get<3>(kv.first);
      if (t == kUnitR) {
        if (a >= P.MT || b >= bwd_rt(P, c)) { printf("R range\n"); return 1; }
        if ((long long)c * P.ldx + b * kBN >= V) { printf("R tile past V\n"); return 1; }
        if (b * kBN + kBN > P.ldx) { printf("R store past the chunk's columns\n"); return 1; }
      } else if (t == kUnitH) {
        if (a >= P.MT || b >= P.NH) { printf("H range\n"); return 1; }
        const int kbs = (bwd_chunk_valid(P, c) + kBK - 1) / kBK;
        if (kbs * kBK > bwd_rt(P, c) * kBN) { printf("H reads unwritten dX columns\n"); return 1; }
        for (int j = 0; j < bwd_rt(P, c); ++j) {
          const long long d = at(kUnitR, c, a, j);
          if (d < 0 || d >= kv.second) { printf("H before its R\n"); return 1; }
        }
      } else {
        const int vt = c == P.NC - 1 ? P.VT_last : P.VT_full;
        if (a >= vt || b >= P.NH) { printf("D range\n"); return 1; }
        if (a * kPairM + kPairM > bwd_rt(P, c) * kBN) { printf("D reads unwritten dX columns\n"); return 1; }
        for (int m = 0; m < P.MT; ++m) {
          const long long d = at(kUnitR, c, m, a);
          if (d < 0 || d >= kv.second) { printf("D before its R\n"); return 1; }
        }
      }
    }
    total += P.total;
  }
  printf("OK %lld\n", total);
  return 0;
}
