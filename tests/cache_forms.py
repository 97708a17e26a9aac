"""Plans that reach every kernel of a paged cache's calls, and the library's own rules (a header without HIP,
compiled here) that say which kernels a call takes."""
import ctypes
import functools
import os
import subprocess
import tempfile

from tests import cache_reference as ref
from tests.op_forms import CSRC

FORMS = ["tokens of 16 rows", "tokens of 32 rows", "rows", "both"]
FEW = 128                                                    # rows up to which waves share a sequence's tokens
SOURCE = """
#include "rc_op_rules.hpp"
extern "C" {
int form(size_t rows, size_t seqs) { return (int)rc::attention_form(rows, seqs); }
int pairs(unsigned d, unsigned rot, int interleaved) { return rc::append_in_pairs(d, rot, interleaved); }
unsigned append(size_t tokens, unsigned rows, unsigned d)
{
    return rc::append_turns(rows, d) / rc::side_by_side(tokens, rc::append_turns(rows, d));
}
unsigned read(size_t tokens, unsigned kv, unsigned d) { return rc::read_turns(kv, d) / rc::side_by_side(tokens, rc::read_turns(kv, d)); }
size_t few() { return rc::kFewRows; }
}
"""


@functools.lru_cache(None)
def rules():
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "rules.cpp"), os.path.join(d, "rules.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib],
                       check=True)
        l = ctypes.CDLL(lib)
    size, word = ctypes.c_size_t, ctypes.c_uint
    l.form.argtypes, l.pairs.argtypes = [size, size], [word, word, ctypes.c_int]
    l.append.argtypes, l.read.argtypes = [size, word, word], [size, word, word]
    l.append.restype = l.read.restype = word
    l.few.restype = size
    return l


def form(plan, group, most=None):
    """The kernels of attention that a plan's call takes."""
    tokens = plan.tokens if not most else min(most, plan.tokens)
    return FORMS[rules().form(tokens * group, len(plan.lengths))]


def by_rows(plan, group, most=None):
    """The sequences whose rows are cut into tiles that waves share by rows."""
    taken = form(plan, group, most)
    return [s for s, n in enumerate(plan.new) if n and (taken == "rows" or taken == "both" and n * group > FEW)]


def by_tokens(plan, group, most=None):
    taken = form(plan, group, most)
    return [s for s, n in enumerate(plan.new) if n and taken != "rows" and (taken != "both" or n * group <= FEW)]


def awkward(page=16):
    """Padding; more rows than tokens; no tokens; a page that is not there in the midst and none at all; a length past
    the table; one token among them. Sequences of 140 rows and more, and of few, of each kind."""
    plan = ref.Plan([(200, 240), (300, 120), (140, -5), (150, 400), (260, 60), (1, 40), (4, 40), (6, 2), (3, -5), (5, 50),
                     (40, 60)], page, seed=4, before=3, behind=9)
    plan.table[0][1] = plan.table[6][1] = plan.pages
    plan.table[3] = plan.table[9] = [-1] * plan.max_pages
    plan.lengths[4] = plan.lengths[10] = 5000
    return plan


def alone(spec, page=16, **more):
    return ref.Plan([spec], page, seed=5, **more)


# what one sequence has that meets the kernel of rows by itself
ALONE = {"whole": (300, 300), "behind": (200, 900), "more rows than tokens": (300, 120), "none": (140, -5)}
MANY_HEADS = [(140, 170), (1, 40)]                           # more heads of the cache than workgroups fit, both kernels
# tokens of the new cases of append and read, and their heads: whole turns and a last one in part
TOKENS = [[(700, 900), (323, 323)], [(700, 900), (324, 330)], [(900, 900), (1, 70), (399, 1000)]]
HEADS = [(32, 16), (36, 9)]
