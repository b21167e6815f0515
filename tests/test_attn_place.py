"""Where attention with shared prefixes finds a token's results: every word that its workspace may hold (of another
call, or of a range that gave up) leads into the slots or nowhere.  The header is compiled and gone through on the host."""
import subprocess

import pytest

from conftest import ROOT

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "%s/speculative_decoding_verify_w4a16_gb300/csrc/attn_place.h"
using namespace w4v;
int main(int, char **argv) {
    const int tok = atoi(argv[1]), group = atoi(argv[2]), ranges = 256, rows = tok * group;
    const size_t slots = 2 * size_t(ranges);
    // every word, as its fields say and with the bits above them set
    for (uint32_t w = 0; w < 1u << 25; ++w) {
        const RowPlace x = read_place(w | (w << 25), ranges, rows, group);
        if (x.parts < 2) continue;                       // 1: at the row's own number; 0: left alone
        for (int k = 0; k < x.parts; k += x.parts - 1)
            for (int head = 0; head < group; head += group > 1 ? group - 1 : 1)
                if (part_slot(x.range, k) * rows + x.tok * group + head >= slots * rows) return printf("%%08x\n", w), 1;
    }
    // the words that are written come back
    for (int range = 0; range < ranges; ++range)
        for (int parts = 0; range + parts <= ranges; ++parts)
            for (int t = 0; t < tok; ++t)
                for (int shares = 0; shares < 2; ++shares) {
                    const RowPlace x = read_place(place_of(range, parts, t, shares != 0), ranges, rows, group);
                    if (x.range != range || x.parts != parts || x.tok != t || x.shares != (shares != 0)) return puts("lost"), 2;
                }
    return 0;
}
""" % ROOT


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("place")
    (d / "place.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-O2", "-std=c++17", str(d / "place.cpp"), "-o", str(d / "place")], check=True)
    return str(d / "place")


@pytest.mark.parametrize("tok,group", [(1, 1), (128, 1), (1, 128), (25, 5), (18, 7), (3, 40), (32, 4), (7, 16)])
def test_every_word_leads_into_the_slots_or_nowhere(program, tok, group):
    r = subprocess.run([program, str(tok), str(group)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
