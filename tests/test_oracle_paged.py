"""Pins of the paged-cache oracle that do not come from its own code."""

import numpy as np
import pytest
import torch

from oracle import paged


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rounding_matches_torch(dtype):
    rng = np.random.default_rng(1)
    x = rng.standard_normal(4096) * 10.0 ** rng.integers(-20, 20, 4096)
    t = torch.from_numpy(x).float().to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    assert np.array_equal(paged.round_to(x, dtype), t.double().numpy())


def test_e4m3_codes_match_torch():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.sort(every[:127]), paged.E4M3)
    rng = np.random.default_rng(2)
    x = np.concatenate([rng.uniform(-448, 448, 4096), rng.uniform(-0.05, 0.05, 4096),
                        (paged.E4M3[1:] + paged.E4M3[:-1]) / 2, [448.0, -448.0, 0.0]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(paged.to_codes(x, "e4m3"), want)


def test_a_quantised_block_is_off_by_at_most_half_a_step():
    rng = np.random.default_rng(3)
    x = paged.round_to(rng.standard_normal((32, 64)), "bf16")
    for fmt in ("e4m3", "int8"):
        c, s = paged.quantise(x, fmt)
        assert np.abs(c).max() == paged.TOP[fmt]
        # half a step: 1/2 of a unit for integers; 2^-4 relative, or half the smallest e4m3 step,
        # 2^-10, plus the fp32 roundings of 1 / amax, the two products and the scale's two (5 * 2^-24 relative)
        half = 0.5 * s if fmt == "int8" else np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s)
        assert (np.abs(c * s - x) <= half + 2.0 ** -21 * np.abs(x)).all()
    assert paged.quantise(np.zeros((32, 64)), "int8")[1] == 0.0


def test_rotation_is_a_rotation_and_relative():
    rng = np.random.default_rng(4)
    a = np.outer(np.arange(9), [0.3, 0.7, 0.01, 1.1])
    cs = np.concatenate([np.cos(a), np.sin(a)], 1)
    for pairs in (False, True):
        x = np.broadcast_to(rng.standard_normal((1, 1, 12)), (9, 1, 12))
        y = np.broadcast_to(rng.standard_normal((1, 1, 12)), (9, 1, 12))
        rx, ry = paged.rotate(x, cs, pairs)[:, 0], paged.rotate(y, cs, pairs)[:, 0]
        assert np.allclose((rx * rx).sum(-1), (x[0] * x[0]).sum())
        assert np.allclose((rx[1:] * ry[:-1]).sum(-1), (rx[1] * ry[0]).sum())
        assert np.array_equal(rx[:, 8:], x[:, 0, 8:])
        assert np.array_equal(rx[0], x[0, 0])
    # one pair by hand: (1, 0) turned by t is (cos t, sin t)
    t = 0.25
    one = np.zeros((1, 1, 2)); one[..., 0] = 1
    got = paged.rotate(one, np.array([[np.cos(t), np.sin(t)]]), True)
    assert np.allclose(got[0, 0], [np.cos(t), np.sin(t)])


def test_attend_against_torch_softmax_and_empty_rows():
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((3, 2, 8)), rng.standard_normal((5, 8)), rng.standard_normal((5, 8))
    out, lse, _, _ = paged.attend(q, k, v)
    x = torch.einsum("igd,td->igt", torch.from_numpy(q), torch.from_numpy(k)) / 8 ** 0.5
    hidden = torch.arange(5) > torch.arange(3)[:, None] + 2
    x = x.masked_fill(hidden[:, None], -torch.inf)
    assert np.allclose(out, (torch.softmax(x, -1) @ torch.from_numpy(v)).numpy())
    assert np.allclose(lse, torch.logsumexp(x, -1).numpy())
    out, lse, _, _ = paged.attend(q, k[:1], v[:1])
    assert not out[:2].any() and np.isneginf(lse[:2]).all()
    assert np.allclose(out[2], v[0])


def test_appending_in_pieces_is_appending_at_once():
    rng = np.random.default_rng(6)
    k, v = rng.standard_normal((2, 100, 16))
    one, many = paged.Head(16, "bf16", "e4m3"), paged.Head(16, "bf16", "e4m3")
    one.append(k, v)
    for a, b in ((0, 1), (1, 31), (31, 32), (32, 97), (97, 97), (97, 100)):
        many.append(k[a:b], v[a:b])
    assert len(one) == len(many) == 100
    for x, y in zip(one.rows(), many.rows()):
        assert np.array_equal(x, y)
