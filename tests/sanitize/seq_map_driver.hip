// Host-side driver of SeqMap (csrc/seq_device.hpp), which says where the sequences
// of a packed batch lie: with right offsets the sequences and their pieces cover
// the rows once each, and with any others (random ones, extremes) every row and every
// slot that the kernels derive from them stays inside the tensors and workspaces.
// Built with AddressSanitizer and UndefinedBehaviorSanitizer on the host side.
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "seq_device.hpp"

using tg::SeqMap;

static int failures = 0;
static void expect(bool ok, const char* what) {
    if (!ok && ++failures < 20) fprintf(stderr, "failed: %s\n", what);
}

static void check(const std::vector<int32_t>& off, int rows, bool right) {
    const int seqs = (int)off.size() - 1;
    const SeqMap m{off.data(), seqs, rows, rows / seqs};
    for (int P : {1, 3, 8, 16, 64}) {
        const int slots = rows / P + seqs;
        std::vector<int> owner(slots, -1), seen(rows, 0);
        for (int s = 0; s < seqs; ++s) {
            const int b = m.start(s), len = m.end(s) - b, first = m.slot0(s, P);
            expect(b >= 0 && len >= 0 && b + len <= rows, "rows in range");
            expect(len == 0 || first + (len - 1) / P < slots, "slots in range");
            expect(first >= 0 && first < slots, "first slot in range");
            for (int slot = 0; slot < slots; ++slot) {  // whatever sequence the search gives
                int lo = -1, hi = -1;
                if (!SeqMap::piece(slot, first, len, P, lo, hi)) continue;
                expect(lo >= 0 && lo <= hi && hi <= len && hi - lo <= P, "piece in range");
                if (!right) continue;
                expect(owner[slot] == -1, "one owner");
                owner[slot] = s;
                for (int l = lo; l < hi; ++l) ++seen[b + l];
            }
        }
        if (right)
            for (int r = 0; r < rows; ++r) expect(seen[r] == 1, "every row once");
    }
}

int main() {
    srand(7);
    const int32_t extreme[] = {INT32_MIN, -1, 0, 1, INT32_MAX, INT32_MAX - 1};
    for (int k = 0; k < 3000; ++k) {
        const int rows = rand() % 200, seqs = 1 + rand() % 9;
        std::vector<int32_t> off(seqs + 1, 0);
        for (int s = 1; s < seqs; ++s) off[s] = rows ? rand() % (rows + 1) : 0;
        off[seqs] = rows;
        std::vector<int32_t> wrong = off;
        for (int s = 1; s < seqs; ++s)
            for (int t = s + 1; t < seqs; ++t)
                if (off[t] < off[s]) std::swap(off[t], off[s]);
        check(off, rows, true);
        for (int32_t& v : wrong)
            if (rand() % 2) v = rand() % 3 ? rand() % (3 * rows + 3) - rows : extreme[rand() % 6];
        check(wrong, rows, false);
        if (rows % seqs == 0) {  // dense
            const SeqMap d{nullptr, seqs, rows, rows / seqs};
            for (int s = 0; s < seqs; ++s)
                expect(d.start(s) == s * d.L && d.end(s) == (s + 1) * d.L &&
                           d.slot0(s, 16) == s * ((d.L + 15) / 16), "dense");
        }
    }
    printf("%d failures\n", failures);
    return failures ? 1 : 0;
}
