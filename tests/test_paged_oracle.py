"""Pins of the paged-cache oracle (CPU): hand-worked plans, closed forms of
the attention, and its invariants."""
import numpy as np
import pytest

from oracle import paged_oracle as P


def test_plan_by_hand():
    # pages of 4 tokens; request 0 holds 3 tokens in page 9 and adds 3: two go
    # to pages of its own; request 1 is idle; request 2 is new with 4 tokens
    table = [[9, -1, -1], [7, 5, -1], [-1, -1, -1]]
    r = P.page_plan([3, 5, 0], [3, 0, 4], table, [2, 4, 6, 8], 1, 4, 9)
    assert r["status"] == 0 and r["used"] == 3
    assert r["table"].tolist() == [[9, 4, -1], [7, 5, -1], [6, -1, -1]]
    assert r["q_offsets"].tolist() == [0, 3, 3, 7] and r["lens"].tolist() == [6, 5, 4]
    assert r["positions"].tolist() == [3, 4, 5, 0, 1, 2, 3, -1, -1]
    assert r["slots"].tolist() == [39, 16, 17, 24, 25, 26, 27, -1, -1]


@pytest.mark.parametrize("lens,new,used,max_tokens,status", [
    ([3], [10], 0, 20, -1),      # beyond the table's 3 pages of 4
    ([-1], [1], 0, 20, -1),
    ([1], [-1], 0, 20, -1),
    ([1], [5], 0, 4, -1),        # more new tokens than the step has room for
    ([1], [1], 5, 20, -1),       # more pages handed out than the list holds
    ([1], [8], 3, 20, -8),       # two pages needed, one left
])
def test_plan_fails_as_a_whole(lens, new, used, max_tokens, status):
    r = P.page_plan(lens, new, [[9, -1, -1]], [1, 2, 3, 4], used, 4, max_tokens)
    assert r["status"] == status and r["used"] == used and r["table"].tolist() == [[9, -1, -1]]
    assert r["lens"].tolist() == lens and set(r["slots"]) == {-1} and r["q_offsets"].tolist() == [0, 0]


def test_attention_closed_forms():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 3, 4, 2, 8))   # [n_pages 3, page 4, Hkv 2, d 8]
    table = np.array([[2, 0, 1]])
    q = np.zeros((1, 4, 8))
    # a zero query weighs all tokens alike: the mean of v, lse = log n
    out, lse, _, _, n = P.attend(q, k, v, table, [10], [0, 1])
    mean = P.gather(v, table[0], np.arange(10)).mean(0)
    assert np.allclose(out[0], np.repeat(mean, 2, 0)) and np.allclose(lse, np.log(10)) and n[0] == 10
    # one visible token: its value, whatever the query
    q = rng.standard_normal((1, 4, 8))
    out, lse, _, _, _ = P.attend(q, k, v, table, [1], [0, 1])
    assert np.allclose(out[0], np.repeat(v[2, 0], 2, 0))
    assert np.allclose(lse[0], [q[0, h] @ k[2, 0, h // 2] / 8 ** 0.5 for h in range(4)])
    # nothing visible
    out, lse, _, _, _ = P.attend(q, k, v, table, [0], [0, 1])
    assert np.all(out == 0) and np.all(lse == -np.inf)
    # a list of every position equals all tokens; a doubled entry counts twice
    q = rng.standard_normal((2, 4, 8))
    every = np.tile(np.arange(12), (2, 1))
    a = P.attend(q, k, v, table, [11], [0, 2])
    b = P.attend(q, k, v, table, [11], [0, 2], idx=every)
    assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1]) and b[4].tolist() == [10, 11]
    c = P.attend(q[:1], k, v, table, [11], [0, 1], idx=np.array([[3, 3, 3, -1, 11]]))
    assert np.allclose(c[0][0], np.repeat(P.gather(v, table[0], [3])[0], 2, 0))


def test_scale_of_a_stored_row():
    assert P.e4m3_scale([[448.0, -1.0], [0.0, 0.0]]).tolist() == [1.0, 2.0 ** -126]
