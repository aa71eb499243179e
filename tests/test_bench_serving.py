"""The cases of bench.py --serving (no GPU needed)."""
import pytest


def test_cases_are_distinct_and_have_work():
    pytest.importorskip("torch")
    import bench
    from perf import operators as ops
    cases = bench.serving_cases(ops)
    assert len({c["name"] for c in cases}) == len(cases) > len(ops.listed())
    for c in cases:
        w = ops.work(c)
        assert w["bytes"] > 0 and w["flops"] >= 0
