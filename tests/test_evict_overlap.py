"""sparse_mla_evict refuses results that overlap its inputs or each other: its CTAs read the inputs while the first
results are written.  Refused on the host, before anything is launched."""

import pytest

import token_sparse_mla_gb300 as smla

# two sequences of three pages into two, 100 rows, a cache of 256 bf16 rows: every argument on a megabyte of its own
SIZES = dict(kv=256 * 1152, tables=2 * 3 * 4, lengths=2 * 4, weights=2 * 192 * 4, new_tables=2 * 2 * 4, kept=2 * 100 * 4, new_lengths=2 * 4,
             new_weights=2 * 128 * 4)
PLACES = {name: (1 + i) << 20 for i, name in enumerate(SIZES)}
RESULTS = ("kept", "new_lengths", "new_weights")
PAIRS = [(a, b) for a in RESULTS for b in SIZES if a != b and not (b in RESULTS and b < a)]


def _refused(**at):
    a = dict(PLACES, **at)
    lib = smla.library()
    st = lib.sparse_mla_evict(a["kv"], a["tables"], a["lengths"], a["weights"], a["new_tables"], 2, 3, 2, 100, 4, 8, 256, 0, a["kept"],
                              a["new_lengths"], a["new_weights"], None)
    return st == 1 and "overlap" in lib.sparse_mla_last_error().decode()


@pytest.mark.parametrize("result,other", PAIRS)
def test_results_that_overlap_are_refused(result, other):
    """The same place, and the last and the first element of one inside the other (16 bytes of the cache)."""
    step = 16 if other == "kv" else 4
    assert _refused(**{result: PLACES[other]})
    assert _refused(**{result: PLACES[other] + SIZES[other] - step})
    assert _refused(**{result: PLACES[other] - SIZES[result] + step})


def test_lengths_are_not_updated_in_place():
    assert _refused(new_lengths=PLACES["lengths"])
    assert _refused(new_weights=PLACES["weights"])
