"""The launch chain of test_pdl_chain with the calls over a paged cache in it.  CPU only.

The page plan and the verification wait first and trigger at their exit.  The paged attention's
first kernel waits, then triggers; the second one of a mixed step triggers at its entry and
reads and writes before its own wait, which it makes before it ends; the merge triggers at its
entry and waits.  So the second kernel's reads and writes have to be safe at its launch: every
earlier kernel that touches the same memory has completed, but for the first kernel of its own
call, with which it shares inputs only."""
import itertools

import pytest

from test_pdl_chain import AFTER_WAIT, CALLS, ENTRY, EXIT, calls, violations

SERVING = ["plan", "paged", "mixed", "verify"]
INPUTS = {"in", "lens", "table", "q_abs", "cache"}


def serving(tag, first_trigger=AFTER_WAIT):
    """Kernels per call: (name, trigger, early reads, writes, early writes)."""
    merge = ("merge", ENTRY, set(), {"out", "out:few", "out:rows"}, set())
    first = ("few", first_trigger, set(), {"partials:few", "out", "out:few"}, set())
    second = ("rows", ENTRY, INPUTS, {"partials:rows", "out", "out:rows"}, {"partials:rows", "out:rows"})
    return {
        "plan": [("plan", EXIT, set(), {"lens", "table", f"slots:{tag}"}, set())],
        "paged": [first, merge],
        "mixed": [first, second, merge],
        "verify": [("verify", EXIT, set(), {"lens", "tokens"}, set())],
    }


# what a kernel reads at any time, for writes made before a wait
READS = {"merge": {"partials:few", "partials:rows"}, "combine": {"partials"}, "split": {"cache", "q_abs", "q_rot"},
         "plan": {"lens", "table"}, "few": INPUTS, "rows": INPUTS, "verify": {"lens", "tokens"}}


def chain(seq, first_trigger=AFTER_WAIT):
    ks = []
    for i, name in enumerate(seq):
        if name in SERVING:
            ks += serving(i, first_trigger)[name]
        else:
            ks += [(*k, set()) for k in calls()(i)[name]]
    return ks


def done_at_launch(ks):
    done = [set() for _ in ks]
    for j in range(1, len(ks)):
        trig = ks[j - 1][1]
        done[j] = set(range(j)) if trig == EXIT else set(range(j - 1)) if trig == AFTER_WAIT else set(done[j - 1])
    return done


def unsafe_writes(ks):
    """(writer, resource, other) where a write before the wait may meet an earlier kernel that
    still reads or writes the same."""
    done, bad = done_at_launch(ks), []
    for j, (name, _, _, _, early) in enumerate(ks):
        for i in range(j):
            touched = ks[i][3] | ks[i][2] | READS.get(ks[i][0], set())
            bad += [(name, r, ks[i][0]) for r in early if r in touched and i not in done[j]]
    return bad


def own_prep(ks, v):
    return ks[v[3]][0] in ("prep", "gqa_prep") and v[0] == v[3] + 1


@pytest.mark.parametrize("length", [1, 2, 3, 4])
def test_early_reads_and_writes_of_the_serving_calls(length):
    names = SERVING + (CALLS if length < 4 else ["append", "absorb", "step"])
    for seq in itertools.product(names, repeat=length):
        ks = chain(seq)
        bad = [v for v in violations([k[:4] for k in ks]) if not own_prep(ks, v)]
        assert not bad, (seq, bad)
        assert not unsafe_writes(ks), (seq, unsafe_writes(ks))


def test_a_first_kernel_that_triggers_at_its_entry_would_race():
    """The second kernel would then write while the merge of the call before still reads its
    partials and writes its rows."""
    for before, res in (("mixed", "partials:rows"), ("paged", "out:rows")):
        bad = unsafe_writes(chain([before, "mixed"], first_trigger=ENTRY))
        assert ("rows", res, "merge") in bad, (before, bad)
        assert not unsafe_writes(chain([before, "mixed"]))
