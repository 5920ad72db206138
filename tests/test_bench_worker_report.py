"""Which worker's failure the multi-process oracle timing quotes."""

import bench


def test_a_workers_own_error_is_quoted_before_the_barrier_it_broke():
    # The failing worker aborts the barrier, so another worker may report the
    # broken barrier first.
    ok = ("ok", 2, 10, 0.0, 1.0)
    broken = ("error", 1, "BrokenBarrierError()", 0.0, 0.0)
    own = ("error", 0, "ValueError('x')", 0.0, 0.0)
    assert bench._first_failure([broken, ok, own]) == own
    assert bench._first_failure([own, broken]) == own
    assert bench._first_failure([broken]) == broken
    assert bench._first_failure([ok]) is None
