// Host-only driver for the order in which attention's workgroups take their tiles,
// built with AddressSanitizer and UndefinedBehaviorSanitizer
// (tests/test_attention_tiles_cpu.py): every tile of every row (or slot) and head is
// one workgroup's, whatever number of units a die takes at a time.
#include <cstdio>
#include <vector>

#include "attn_internal.h"

using namespace wkv7::attn;

namespace {
int g_fails = 0, g_cut = 0, g_many = 0;

// ids 0 .. slots heads - 1 against (slot, head), each once; later workgroups of a unit
// have no more to go over than earlier ones.
void check(const Seqs &m, int64_t B, int64_t heads, uint32_t chunk, bool last_first)
{
    const int64_t n = m.slots * heads;
    std::vector<char> seen(n, 0);
    std::vector<int> before(B * heads, -1);
    for (int64_t id = 0; id < n; ++id) {
        int slot = -1, head = -1;
        unit_of(m, B, heads, chunk, last_first, (uint32_t)id, slot, head);
        if (slot < 0 || slot >= m.slots || head < 0 || head >= heads || seen[slot * heads + head]++) {
            std::fprintf(stderr, "B %ld heads %ld tiles %ld slots %ld chunk %u packed %d: id %ld -> slot %d head %d\n", (long)B,
                         (long)heads, (long)m.tiles, (long)m.slots, chunk, m.starts != nullptr, (long)id, slot, head);
            ++g_fails;
            return;
        }
        const int64_t row = m.starts ? 0 : slot / m.tiles;
        const int tile = (int)(m.starts ? slot : slot % m.tiles), at = last_first ? -tile : tile;
        int &was = before[row * heads + head];
        if (was != -1 && at <= (last_first ? -was : was)) {
            std::fprintf(stderr, "order: B %ld heads %ld tiles %ld chunk %u id %ld\n", (long)B, (long)heads, (long)m.tiles,
                         chunk, (long)id);
            ++g_fails;
            return;
        }
        was = tile;
    }
    const int64_t units = m.starts ? heads : B * heads;
    if (units % 8 == 0 && chunk < units / 8) {
        ++g_many;
        if (units / 8 % chunk) ++g_cut;
    }
}

Seqs rows(int64_t B, int64_t T)
{
    const int64_t tiles = (T + kTile - 1) / kTile;
    return {nullptr, T, B, tiles, B * tiles};
}
}  // namespace

int main()
{
    static const int32_t kStarts[2] = {0, 0};
    for (int64_t B : {1, 2, 3, 5, 9, 17})
        for (int64_t heads : {1, 2, 3, 8, 11, 16, 40})
            for (int64_t T : {1, 128, 129, 300, 1025})
                for (bool last_first : {false, true}) {
                    const Seqs m = rows(B, T);
                    for (uint32_t chunk : {1u, 2u, 3u, 5u, 7u, 8u, 64u, 1000u}) {
                        check(m, B, heads, chunk, last_first);
                        check(narrow(m, B), B, heads, chunk, last_first);
                    }
                    Seqs p = m;   // packed: B sequences in T tokens
                    p.starts = kStarts;
                    p.nseq = B;
                    p.slots = T / kTile + B;
                    for (uint32_t chunk : {1u, 2u, 5u, 1000u}) {
                        check(p, 1, heads, chunk, last_first);
                        check(narrow(p, 1), 1, heads, chunk, last_first);
                    }
                }
    // as the launches have it: rows long enough that a die takes its units in turns
    g_cut = g_many = 0;
    for (int64_t D : {64, 128})
        for (int64_t size : {2, 4})
            for (int64_t T : {1025, 2050, 4096, 9000, 70000})
                for (int64_t B : {1, 3, 8, 17})
                    for (int64_t Hk : {1, 5, 8, 24})
                        for (int64_t group : {1, 4, 8}) {
                            const int64_t Hq = Hk * group, bytes = T * 2 * D * size;
                            const Seqs m = rows(B, T);
                            if (m.slots * Hq > 200000) continue;
                            check(m, B, Hq, chunk_of(m, B * Hq, bytes, group), true);
                            check(m, B, Hk, chunk_of(m, B * Hk, bytes * group, 1), false);
                        }
    if (g_many < 50 || g_cut < 10) {
        std::fprintf(stderr, "%d launches in turns, %d with a last one that is cut: too few\n", g_many, g_cut);
        ++g_fails;
    }
    if (g_fails) std::fprintf(stderr, "%d checks failed\n", g_fails);
    return g_fails != 0;
}
