"""Sizes at the ends of what the cache and attention calls take, on the CPU: a
refused call returns its status before any device call."""
import pytest

import int4_dequantize_matmul_amd as q4
from tests.test_serving_host import APPEND, SH, cache, call

TOP = 2 ** 63 - 1


def test_workgroups_of_the_queries_count():
    """Two of each of T / 16 + 2 sequences and head, and one of each started 16 rows and query head: together below 2^32."""
    N = 3 * 2 ** 28
    big = dict(APPEND, cache=cache(heads=1, sequences=N, table=1), T=1, Hq=2 ** 31 - 1, q_token=0)
    assert call("q8_kv_append", big) == SH
    # 17 rows are two times 16
    assert call("q8_kv_append", dict(big, T=17, Hq=2 ** 26, cache=cache(heads=1, sequences=2 ** 30 - 2 ** 25, table=1))) == SH


@pytest.mark.parametrize("window,sinks", [(TOP, 0), (TOP, 1), (TOP - 31, 0), (1, TOP), (2 ** 62, 2 ** 62), (TOP, TOP),
                                          (131072, 0), (2 ** 40, 2 ** 40)])
def test_windows_past_every_length_share_the_keys_like_none(window, sinks):
    f = q4.q8_attention_workspace
    none = f(1, 1, 32, 8, 128, 131072)
    assert none > 0 and f(1, 1, 32, 8, 128, 131072, window, sinks) == none
    assert f(1, 1, 32, 8, 128, 131072, 1000, 4) < none
