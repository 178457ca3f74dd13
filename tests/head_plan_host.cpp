// Host-side check of the loss's workspace (csrc/head_plan.h): over rows, vocabularies, widths, both types, both
// alignments and several numbers of SMs, every region holds what the launches write there, by the same functions
// that the launches choose by, and a workspace of more rows holds every smaller call.
// Prints the first violations of each kind and a count; exit status 0 = none.
#include <cstdio>
#include <vector>

#include "head_plan.h"

using namespace oomb::head;

static long bad = 0, checked = 0;
static void need(const char* what, bool holds, int64_t n, int D, int V, int dtype, bool on16, int sms, size_t want, size_t has) {
  ++checked;
  if (holds) return;
  if (++bad <= 20)
    std::printf("%s: n %lld D %d V %d %s%s, %d SMs: %zu bytes of %zu\n", what, (long long)n, D, V, dtype ? "fp32" : "bf16",
                on16 ? "" : " off 16 bytes", sms, want, has);
}

static void one(int64_t n, int D, int V, int dtype, bool on16, int sms) {
  const int clusters = sms / 2;
  {
    const Plan p = make_plan(n, D, V, dtype, false, on16, clusters);
    const size_t given = make_plan(n, D, V, dtype, false, true, clusters).bytes;  // what a caller asks for
    const RowParts r = row_parts(n, V, p.piece, clusters);
    const size_t want = (size_t)n * r.parts * 8;
    need("parts of the row sums", p.part + want <= given, n, D, V, dtype, on16, sms, want, given - p.part);
    need("gathered rows", p.x + (size_t)n * p.parts_of * p.pitch_d * 2 <= p.w, n, D, V, dtype, on16, sms, 0, 0);
    if (p.staged) {
      const size_t w = (size_t)p.piece * p.parts_of * p.pitch_d * 2;
      need("staged rows of W", p.w + w <= p.part, n, D, V, dtype, on16, sms, w, p.part - p.w);
    }
    // a piece ends where the next one's first part begins
    need("whole parts a piece", p.piece == V || p.piece % kTile == 0, n, D, V, dtype, on16, sms, p.piece, V);
  }
  {
    const Plan p = make_plan(n, D, V, dtype, true, on16, clusters);
    const size_t given = make_plan(n, D, V, dtype, true, true, clusters).bytes;
    const size_t z = (size_t)p.parts_of * n * p.pitch_z * 2, pitch = up((size_t)D, 4);
    need("dz", p.dz + z <= p.acc, n, D, V, dtype, on16, sms, z, p.acc - p.dz);
    const size_t acc = (size_t)most_splits(n, D) * n * pitch * 4;
    need("sums of dx", p.acc + acc <= p.acc_w, n, D, V, dtype, on16, sms, acc, p.acc_w - p.acc);
    for (int cols : {p.piece, V - (V - 1) / p.piece * p.piece}) {
      const int splits = dw_splits(n, D, cols, clusters);
      const size_t w = splits > 1 ? (size_t)splits * cols * pitch * 4 : 0;
      need("sums of dw", p.acc_w + w <= given, n, D, V, dtype, on16, sms, w, given - p.acc_w);
    }
    if (p.staged) {
      const size_t w = (size_t)p.piece * p.parts_of * p.pitch_d * 2;
      need("staged rows of W, backward", p.w + w <= p.dz, n, D, V, dtype, on16, sms, w, p.dz - p.w);
    }
    need("a forward in a backward's workspace", make_plan(n, D, V, dtype, false, true, clusters).bytes <= given, n, D, V,
         dtype, on16, sms, 0, given);
  }
}

int main() {
  std::vector<int> rows, vocabularies;
  for (int n = 1; n <= 70; ++n) rows.push_back(n);
  for (int t = 256; t <= 256 * 80; t += 256)  // a tile's last row and the next tile's first
    for (int e : {-1, 0, 1}) rows.push_back(t + e);
  for (int n : {77, 300, 777, 3000, 30011, 70001, 131072, 1000003, 20000001}) rows.push_back(n);
  std::sort(rows.begin(), rows.end());
  for (int v = 1; v <= 6200; v += v < 700 ? 1 : 13) vocabularies.push_back(v);
  for (int v : {512, 1100, 2316, 2400, 32001, 50001, 57899, 131072, 600001, 5000000}) vocabularies.push_back(v);
  for (int sms : {2, 40, 148, 152})
    for (int dtype : {OOMB_BF16, OOMB_FP32})
      for (int D : {1, 264, 1000, 3584, 20000}) {
        if (sms < 148 && D != 264) continue;
        for (int V : vocabularies) {
          size_t last[2] = {0, 0};
          for (int n : rows) {
            for (bool on16 : {true, false}) one(n, D, V, dtype, on16, sms);
            for (int b : {0, 1}) {
              const size_t bytes = make_plan(n, D, V, dtype, b != 0, true, sms / 2).bytes;
              need(b ? "grows with n, backward" : "grows with n", bytes >= last[b], n, D, V, dtype, true, sms, last[b], bytes);
              last[b] = bytes;
            }
          }
        }
      }
  std::printf("%ld of %ld do not hold\n", bad, checked);
  return bad != 0;
}
