"""The cache's oracle against cases worked out by hand."""
import numpy as np

from oracle import kv_cache_oracle as kvo


def test_plan():
    table = np.full((3, 3), -1, np.int32)
    table[0, 0], table[2, :2] = 7, [4, 9]
    free = np.array([1, 3, 5, 6, 8], np.int32)
    got = kvo.plan(np.array([2, 0, 15], np.int32), np.array([15, 0, 18], np.int32), table, free, 1, 16, 19)
    status, lens, taken, cu, pos, slots, after = got
    assert (status, list(lens), taken, list(cu)) == (0, [17, 0, 33], 3, [0, 2, 2, 17])
    assert list(pos[:3]) == [15, 16, 18] and list(slots[:3]) == [7 * 16 + 15, 3 * 16, 9 * 16 + 2]
    assert slots[16] == 5 * 16 and list(slots[17:]) == [-1, -1] and after[0, 1] == 3 and after[2, 2] == 5
    for kw, bit in ((dict(taken=4), 1), (dict(rows=16), 4), (dict(add=np.array([40, 0, 0], np.int32)), 2),
                    (dict(add=np.array([-1, 0, 0], np.int32)), 8)):
        a = dict(add=np.array([2, 0, 15], np.int32), taken=1, rows=19) | kw
        got = kvo.plan(a["add"], np.array([15, 0, 18], np.int32), table, free, a["taken"], 16, a["rows"])
        assert got[0] & bit and (got[6] == table).all() and (got[5] == -1).all() and not got[3].any()


def test_write_moves_what_was_there():
    codes, most = np.zeros((2, 1, 16, 2), np.int8), np.zeros((2, 1))
    codes, most = kvo.write(np.array([[[1.0, -2.0]], [[0.5, 0.0]]]), [16, 17], codes, most)
    assert most[1, 0] == 2 and codes[1, 0, :2].tolist() == [[64, -127], [32, 0]]  # 63.5 and 31.75; a half goes to even
    codes, most = kvo.write(np.array([[[4.0, 1.0]]]), [18], codes, most)
    assert most[1, 0] == 4 and codes[1, 0, :3].tolist() == [[32, -64], [16, 0], [127, 32]]
    codes, most = kvo.write(np.array([[[1.0, 0.0]]]), [16], codes, most)  # a block begun anew
    assert most[1, 0] == 1 and codes[1, 0, 0].tolist() == [127, 0]


def test_attn_is_a_softmax_over_what_a_row_sees():
    rng = np.random.default_rng(0)
    Kc, Vc = (rng.integers(-127, 128, (4, 1, 16, 8)).astype(np.int8) for _ in range(2))
    one = np.full((4, 1), 127.0)
    q = rng.standard_normal((2, 2, 8)) * 0.01
    O, A, _ = kvo.attn(q, Kc, Vc, one, one, np.array([2, 0]), 18, 1.0)
    K, V = np.concatenate([Kc[2, 0], Kc[0, 0]]).astype(float), np.concatenate([Vc[2, 0], Vc[0, 0]]).astype(float)
    for i, n in ((0, 17), (1, 18)):
        w = np.exp(q[i] @ K[:n].T)
        np.testing.assert_allclose(O[i], w @ V[:n] / w.sum(1, keepdims=True), rtol=1e-12, atol=1e-12)
    O, _, _ = kvo.attn(q, Kc, Vc, one, one, np.array([2, 0]), 1, 1.0)
    assert (O[0] == 0).all() and (O[1] == V[0]).all()
