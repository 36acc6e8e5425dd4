"""Sizes at the ends of what the cache and attention calls take, on the CPU: a
refused call returns its status before any device call."""
from tests.test_serving_host import APPEND, SH, cache, call


def test_workgroups_of_the_queries_count():
    """Two of each of T / 16 + 2 sequences and head, and one of each started 16 rows and query head: together below 2^32."""
    N = 3 * 2 ** 28
    big = dict(APPEND, cache=cache(heads=1, sequences=N, table=1), T=1, Hq=2 ** 31 - 1, q_token=0)
    assert call("q8_kv_append", big) == SH
    # 17 rows are two times 16
    assert call("q8_kv_append", dict(big, T=17, Hq=2 ** 26, cache=cache(heads=1, sequences=2 ** 30 - 2 ** 25, table=1))) == SH
