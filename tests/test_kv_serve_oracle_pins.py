"""Hand-derived results of the oracle of 4-bit caches, verification and eviction."""

import numpy as np

from oracle import kv_serve_ref as ref


def test_scales():
    assert ref.scale_of(7.0, False) == 1.0 and ref.scale_of(0.0, False) == 0.0
    assert ref.scale_of(7 * 1.03125, False) == 1.0       # 33 / 32: a tie, to the even 16 / 16
    assert ref.scale_of(7 * 1.09375, False) == 1.125     # 35 / 32: a tie, to the even 18 / 16
    assert ref.scale_of(7 * 1.9999, False) == 2.0
    assert ref.scale_of(7 * 2.0**-101, False) == 0.0 and ref.scale_of(7 * 2.0**-101, True) == 0.0
    assert ref.scale_of(65504.0, True) == 9216.0 and ref.scale_of(3.0e38, False) == 2.0**121
    assert ref.scale_of(7 * 2.0**-24, True) == 2.0**-24


def test_codes():
    x = np.zeros(64)
    x[:6] = [7, -7, 0.5, 1.5, -2.5, 3.49]
    x[32:35] = [14, 1, -3]
    codes, scales = ref.quantise(x, False)
    assert scales.tolist() == [1.0, 2.0]
    assert codes[:6].tolist() == [15, 1, 8, 10, 6, 11] and codes[32:35].tolist() == [15, 8, 6]  # ties to even
    packed = ref.pack(codes)
    assert packed[0] == 15 | 1 << 4 and packed[1] == 8 | 10 << 4 and packed.shape == (32,)
    assert ref.values(packed, scales)[:6].tolist() == [7, -7, 0, 2, -2, 3]
    x[3] = np.inf
    codes, scales = ref.quantise(x, False)
    assert np.isnan(scales[0]) and scales[1] == 2 and (codes[:32] == 8).all()


def rows(*r):
    return np.array([r], np.float32)


def test_verify_chain():
    p = rows([0.5, 0.5, 0, 0], [0, 0.25, 0.75, 0], [0, 0, 0, 1])
    q = rows([1, 0, 0, 0], [0, 0, 0.875, 0.125])
    tokens = np.array([[0, 2]], np.int32)
    u = np.array([[0.4, 0.9, 0.5]], np.float32)
    # 0.4 < 0.5: accepted; 0.9 * 0.875 = 0.7875 >= 0.75: rejected, what is left is token 1 alone
    got = ref.verify(p, tokens, u, q)
    assert got[0].tolist() == [[0, -1]] and got[1].tolist() == [1] and got[2].tolist() == [1] and not got[3]
    u[0, 1] = 0.85  # 0.74375 < 0.75: both, and the last row draws
    assert ref.verify(p, tokens, u, q)[2].tolist() == [3]
    u[0, 0] = 0.5   # 0.5 < 0.5 is false: the rest of the first row is token 1
    got = ref.verify(p, tokens, u, q)
    assert got[1].tolist() == [0] and got[2].tolist() == [1]


def test_verify_siblings_and_draw():
    p = rows([0.5, 0.25, 0.25], [1, 0, 0], [0, 1, 0], [0, 0, 1])
    tokens, parents = np.array([[0, 1, 2]], np.int32), np.array([[-1, -1, -1]], np.int32)
    # certain tokens: 0 with 1/2; of the rest (1/2, 1/2) token 1 with 1/2; token 2 for certain
    for u, path, token in ([0.49, 0, 0, 0], 0, 0), ([0.5, 0.49, 0, 0], 1, 1), ([0.5, 0.5, 0.99, 0], 2, 2):
        got = ref.verify(p, tokens, np.array([u], np.float32), None, parents)
        assert got[0].tolist() == [[path, -1, -1]] and got[2].tolist() == [token]
    got = ref.verify(p, tokens[:, :0], np.array([[0.75]], np.float32))
    assert got[2].tolist() == [2]  # running sums 1/2, 3/4, 1: 3/4 is not above 3/4
    got = ref.verify(p * 0, tokens[:, :0], np.array([[0.75]], np.float32))
    assert got[2].tolist() == [-1] and got[3]


def test_evict():
    w = np.array([[5, 1, 4, 4, 0, 9, 2]], np.float32)
    path, n_draft, n_keep, out = ref.evict(w, [7], 4, 1, 1)
    assert path.tolist() == [[0, 2, 5, 6]] and n_draft.tolist() == [7] and n_keep.tolist() == [4]
    assert out.tolist() == [[5, 4, 9, 2, 0, 0, 0]]
    path, n_draft, n_keep, out = ref.evict(w, [4], 4, 1, 1)
    assert (path == -1).all() and n_draft.tolist() == [0] and out.tolist() == [[5, 1, 4, 4, 0, 0, 0]]


def test_weigh():
    keys = np.zeros((1, 1, 4, 32))
    keys[0, 0, :, 0] = [0, np.log(2), np.log(3), np.log(4)]
    q = np.zeros((1, 2, 1, 32))
    q[..., 0] = 1
    lse = np.log(np.array([[[6.0], [10.0]]]))
    out, _ = ref.weigh(q, keys, np.array([[0]]), [4], lse, np.array([[8.0, 8, 8, 8, 7]]), scale=1.0, decay=0.5)
    assert np.allclose(out, [[4 + 1 / 6 + 0.1, 4 + 1 / 3 + 0.2, 0.5 + 0.3, 0.4, 7]])
